"""Training steps of one MoE block on the symmetric heap.

    python examples/train_moe_block.py [--steps 20] [--config tiny|mixtral] [--tokens-per-slot 512] [--inter 4096]

The block is  y = x + scale * drop(tanh(gate) * norm(MoE(norm(x)))).  Its
forward dispatches the normalised tokens over the heap, runs the experts as
grouped products with the routing weight inside the SwiGLU, and combines
without weights.  Its backward is made of the same pieces turned around: the
combine's backward is a dispatch of the output's gradient (same routing, so the
same rows), the dispatch's backward is an unweighted combine.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import combine_symmetric_heap_gb300 as sm  # noqa: E402
import moe_synth as ms  # noqa: E402


class MoeBlock:
    """One block's parameters (bf16), its two heaps and what the backward needs.

    ``gate_up`` holds each expert's gate rows above its up rows, so that both
    are one grouped product, forward and backward.
    """

    def __init__(self, cfg: dict, scale: float = 0.5, dropout: float = 0.1, seed: int = 0, device="cuda"):
        W, H, I, E, k = (cfg[n] for n in ("world", "hidden", "inter", "num_experts", "topk"))
        self.cfg, self.scale, self.p, self.seed, self.step = cfg, scale, dropout, seed, 0
        self.n, self.k = W * cfg["tokens_per_slot"], k
        self.heap = sm.SymHeap(cfg, device)        # the forward's rows, kept for the backward
        self.grad_heap = sm.SymHeap(cfg, device)   # the gradients' rows, in the same layout
        wg, wu, wd = ms.weights_torch(cfg, device)
        bf = dict(device=device, dtype=torch.bfloat16)
        self.params = {
            "norm_in": torch.ones(H, **bf), "norm_out": torch.ones(H, **bf),
            "gate": torch.full((1, H), 0.5, **bf),
            "router": (0.02 * torch.randn(E, H, device=device, generator=torch.Generator(device).manual_seed(seed))).bfloat16(),
            "gate_up": torch.cat((wg.view(E, I, H), wu.view(E, I, H)), 1), "down": wd.view(E, H, I).clone(),
        }
        self.grads = {name: torch.empty_like(t) for name, t in self.params.items()}
        tokens, rows = (self.n, H), (W, self.heap.cap)
        self.h, self.out, self.do, self.dh, self.dh_router = (torch.empty(tokens, **bf) for _ in range(5))
        self.logits = torch.empty(self.n, E, device=device)
        self.idx = torch.empty(self.n, k, dtype=torch.int32, device=device)
        self.w = torch.empty(self.n, k, device=device)
        self.gu, self.dgu = torch.empty(*rows, 2 * I, **bf), torch.empty(*rows, 2 * I, **bf)
        self.d_hidden = torch.empty(*rows, I, **bf)
        self.d_row_w = torch.empty(rows, device=device)
        self.rstd_in, self.rstd_out = torch.empty(self.n, device=device), torch.empty(self.n, device=device)
        # all tokens as one group, for the router's products
        self.all = dict(cnt=torch.tensor([self.n], dtype=torch.int32, device=device),
                        off=torch.zeros(1, dtype=torch.int32, device=device))
        self.work = torch.empty(sm.moe_block_norm_workspace(self.n, H, 1), dtype=torch.uint8, device=device)

    def _groups(self):
        win = self.heap.window
        return dict(cnt=win("cnt"), off=win("recv_off"), status=self.heap.status_word())

    def _end(self):
        """The norm after the block with gate, dropout and scale."""
        q = self.params
        return dict(o=self.out, w_post=q["norm_out"], gate=q["gate"], gate_act="tanh", scale=self.scale, p=self.p,
                    seed=self.seed, offset=self.step, rstd_post=self.rstd_out)

    def forward(self, x, y):
        q, heap, win, I = self.params, self.heap, self.heap.window, self.cfg["inter"]
        self.x = x
        sm.moe_block_norm(x, w_pre=q["norm_in"], h=self.h, rstd_pre=self.rstd_in)
        heap.router_logits(self.h, q["router"], self.logits)
        heap.route_topk(self.logits, self.idx, self.w)
        heap.dispatch(self.h, self.idx, self.w)
        sm.moe_grouped_matmul(win("recv_x"), q["gate_up"], out=self.gu, **self._groups())
        sm.moe_swiglu_rows(self.gu[..., :I], self.gu[..., I:], win("h"), row_w=win("recv_w"), total=win("total"))
        sm.moe_grouped_matmul(win("h"), q["down"], out=win("y"), **self._groups())
        heap.combine(self.idx, None, self.out, unweighted=True)
        sm.moe_block_norm(x, y=y, **self._end())

    def backward(self, dy, dx):
        """Gradients of the parameters into ``grads``, of x into dx."""
        q, d, heap, back, I = self.params, self.grads, self.heap, self.grad_heap, self.cfg["inter"]
        win, bwin, groups = heap.window, back.window, self._groups()
        sm.moe_block_norm_bwd(dy=dy, do=self.do, dw_post=d["norm_out"], dgate=d["gate"], work=self.work, **self._end())
        back.dispatch(self.do, self.idx, self.w)  # the combine's backward: each row gets its token's gradient
        rows = bwin("recv_x")
        sm.moe_grouped_wgrad(rows, win("h"), dw=d["down"], **groups)
        sm.moe_grouped_matmul(rows, q["down"], out=self.d_hidden, trans_w=True, **groups)
        sm.moe_swiglu_rows_bwd(self.gu[..., :I], self.gu[..., I:], self.d_hidden, self.dgu[..., :I], self.dgu[..., I:],
                               row_w=win("recv_w"), d_row_w=self.d_row_w, total=win("total"))
        sm.moe_grouped_wgrad(self.dgu, win("recv_x"), dw=d["gate_up"], **groups)
        sm.moe_grouped_matmul(self.dgu, q["gate_up"], out=bwin("y"), trans_w=True, **groups)
        back.combine(self.idx, None, self.dh, unweighted=True)  # the dispatch's backward: a token's rows summed
        # router: the rows' weight gradients back to their tokens, through the softmax over the chosen k
        pos = torch.cat([heap.pos(s) for s in range(self.cfg["world"])]).long()
        slot = self.idx.long() // (self.cfg["num_experts"] // self.cfg["world"])
        dw = self.d_row_w[slot, pos]
        dsel = self.w * (dw - (self.w * dw).sum(1, keepdim=True))
        experts = self.cfg["num_experts"]
        wide = torch.zeros(self.n, -(-experts // 8) * 8, device=dsel.device, dtype=torch.bfloat16)  # 16-byte rows
        dlogits = wide.scatter_(1, self.idx.long(), dsel.bfloat16())[:, :experts]
        sm.moe_grouped_wgrad(dlogits, self.h, dw=d["router"][None], **self.all)
        sm.moe_grouped_matmul(dlogits, q["router"][None], out=self.dh_router, trans_w=True, **self.all)
        self.dh += self.dh_router
        sm.moe_block_norm_bwd(dy=dy, dh=self.dh, y=self.x, w_pre=q["norm_in"], rstd_pre=self.rstd_in, dx=dx,
                              dw_pre=d["norm_in"], work=self.work)

    def update(self, lr: float):
        for name, t in self.params.items():
            t -= lr * self.grads[name]
        self.step += 1  # another dropout mask


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--config", default="tiny", choices=("tiny", "mixtral"))
    ap.add_argument("--tokens-per-slot", type=int, help="instead of the configuration's")
    ap.add_argument("--inter", type=int, help="expert intermediate size, instead of the configuration's")
    ap.add_argument("--lr", type=float, default=0.5)
    a = ap.parse_args()
    cfg = ms.shape_of(ms.CONFIGS[a.config])
    cfg.update({k: v for k, v in (("tokens_per_slot", a.tokens_per_slot), ("inter", a.inter)) if v})
    dev = torch.device("cuda", torch.cuda.current_device())
    block = MoeBlock(cfg, device=dev)
    x = ms.x_torch(cfg, dev)
    gen = torch.Generator(dev).manual_seed(1)
    target = x + 0.5 * torch.randn(x.shape, generator=gen, device=dev).bfloat16()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    first = None
    for step in range(a.steps):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        block.forward(x, y)
        diff = y.float() - target.float()
        loss = diff.square().mean()
        # the gradient of the mean, times the tokens: one learning rate for every size
        block.backward((2 / x.shape[1] * diff).bfloat16(), dx)
        end.record()
        block.update(a.lr / x.shape[0])
        first = float(loss) if first is None else first
        print(f"step {step}: loss {float(loss):.5f}, forward and backward {start.elapsed_time(end):.3f} ms")
    assert block.heap.status() == 0 and block.grad_heap.status() == 0
    return first, float(loss)


if __name__ == "__main__":
    main()
