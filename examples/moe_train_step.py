"""Training steps of a mixture-of-experts layer with 8-bit products.

One linear map per expert: y[t] = sum over the chosen experts e of w[t][e] W[e] x[t],
trained by plain gradient descent towards a fixed random teacher. Every step goes
through the library: routing with the balance loss, the experts' products, the
experts' weight gradients, the router's gradient, and one clipping of all
gradients together. Gathers, the router's two small products and the update
are torch's.

With score="sigmoid" (or "softmax") the router goes by scores plus a bias that
evens out the experts' loads; with adamw the update is the library's AdamW step,
which clips by itself, states in 32 or 8 bits; serve() answers through products in
8-bit integers.

    python examples/moe_train_step.py [--steps 30] [--score sigmoid] [--adamw 8]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_quantizer_amd as fp8g  # noqa: E402


def _pad(n):
    return (n + 127) // 128 * 128


class MoELayer:
    """Parameters (fp32) and the buffers that every step uses again."""

    def __init__(self, tokens, width, out, experts, top_k, balance=0.01, device="cuda", seed=0, score=None,
                 groups=1, open_groups=1, adamw=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.T, self.K, self.N, self.E, self.k, self.balance = tokens, width, out, experts, top_k, balance
        new = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=device)  # noqa: E731
        self.router = torch.randn(experts, width, device=device, generator=g) * width ** -0.5
        self.weight = torch.randn(experts, out, width, device=device, generator=g) * width ** -0.5
        # as many rows as the contiguous layout can need, known without asking the device
        self.rows = _pad(tokens * top_k + experts * 127)
        R, i32, u8, bf16 = self.rows, torch.int32, torch.uint8, torch.bfloat16
        self.route = dict(expert_ids=new(tokens, top_k, dtype=i32), weights=new(tokens, top_k),
                          counts=new(experts, dtype=i32), routed=new(1, dtype=i32), prob_sum=new(experts),
                          loss=new(1), group_offsets=new(experts + 1, dtype=i32), slots=new(tokens, top_k, dtype=i32))
        self.route_ws = new(max(16, fp8g.moe_route_workspace_size(tokens, experts)), dtype=u8)
        self.qx, self.sx = new(R, width, dtype=u8), new(width // 128, R)
        self.qw, self.sw = new(experts, out, width, dtype=u8), new(experts, out // 128, width // 128)
        self.y = new(R, out, dtype=bf16)
        # operands of the weight gradient: tokens last
        self.qa, self.sa = new(out, R, dtype=u8), new(R // 128, out, dtype=u8)
        self.qb, self.sb = new(width, R, dtype=u8), new(R // 128, width, dtype=u8)
        self.d_weight = new(experts, out, width, dtype=bf16)
        self.sumsq, self.norm, self.one = new(1, dtype=torch.float64), new(1), torch.ones(1, device=device)
        self.clip_ws = new(max(8, fp8g.grad_norm_sq_workspace_size([self.d_weight, self.router])), dtype=u8)
        # routing by scores: what its two calls share, and the choice's bias
        self.scored = score and dict(score=score, renormalise=True, loss_coef=balance)
        self.choice = dict(groups=groups, open_groups=open_groups, group_best=min(2, experts // groups))
        self.bias = torch.zeros(experts, device=device)
        self.adamw, self.steps = adamw, 0
        if adamw:
            params, self.d_router = [self.weight, self.router], new(experts, width)
            fresh = lambda f: [f(p.numel()) for p in params]  # noqa: E731
            zeros = lambda n, dtype=torch.float32: torch.zeros(n, dtype=dtype, device=device)  # noqa: E731
            code, block = (lambda n: zeros(n, u8)), (lambda n: zeros(-(-n // 128), u8))
            states = [fresh(code if adamw == 8 else zeros) for _ in range(2)]
            scales = dict(m_scales=fresh(block), v_scales=fresh(block)) if adamw == 8 else {}
            self.states = states + list(scales.values())
            self.tensors = fp8g.adamw_tensors(params, [self.d_weight, self.d_router], *states, **scales)

    def _route(self, x, mask):
        """Rows of the experts' operand, filled; each pair's row of it."""
        r = self.route
        self.logits = x.float() @ self.router.t()
        if self.scored:
            fp8g.moe_route_scored(self.logits, self.k, *r.values(), self.route_ws, bias=self.bias, token_mask=mask,
                                  **self.scored, **self.choice)
        else:
            fp8g.moe_route(self.logits, self.k, *r.values(), self.route_ws, token_mask=mask, renormalise=True,
                           loss_coef=self.balance)
        live = r["slots"] >= 0
        # (rows that no token fills stay zero; a pair without a slot goes to a
        # spare row past the end)
        self.at = torch.where(live, r["slots"], self.rows).long()
        self.xr = torch.zeros(self.rows + 1, self.K, dtype=torch.bfloat16, device=x.device)
        self.xr[self.at.reshape(-1)] = x.repeat_interleave(self.k, 0)
        self.xr = self.xr[: self.rows]
        self.w = torch.where(live, r["weights"], torch.zeros_like(r["weights"]))

    def forward(self, x, mask=None):
        """x bf16 [T][K] -> y fp32 [T][N]; keeps what the backward pass needs."""
        self._route(x, mask)
        fp8g.fp8_quantize_bf16(self.xr, 1, self.qx, self.sx, 1, self.rows)
        fp8g.fp8_quantize(self.weight.view(-1, self.K), 128, self.qw.view(-1, self.K),
                          self.sw.view(-1, self.K // 128), self.K // 128, 1)
        self.y.zero_()
        fp8g.grouped_gemm_fp8_contiguous(self.qx, self.sx, self.qw, self.sw, self.y, self._all_rows())
        return self._combine()

    def _combine(self):
        self.picked = torch.cat([self.y, self.y.new_zeros(1, self.N)])[self.at].float()   # [T][k][N]
        return (self.w[..., None] * self.picked).sum(1)

    def freeze(self):
        """The weights' int8 codes and scales for serve."""
        self.iw = torch.empty(self.weight.shape, dtype=torch.int8, device=self.weight.device)
        self.siw = torch.empty(self.weight.shape[:2], device=self.weight.device)
        fp8g.int8_quantize(self.weight.view(-1, self.K), self.iw.view(-1, self.K), self.siw.view(-1))
        self.ix = torch.empty(self.rows, self.K, dtype=torch.int8, device=self.weight.device)
        self.six = torch.empty(self.rows, device=self.weight.device)

    def serve(self, x, mask=None):
        """x bf16 [T][K] -> y fp32 [T][N] by products in 8-bit integers."""
        self._route(x, mask)
        fp8g.int8_quantize(self.xr, self.ix, self.six)
        self.y.zero_()
        fp8g.grouped_gemm_int8_contiguous(self.ix, self.six, self.iw, self.siw, self.y, self.route["group_offsets"])
        return self._combine()

    def _all_rows(self):
        """The offsets as the product wants them: the last expert's rows reach
        the end of the operand (the spare ones are zero)."""
        off = self.route["group_offsets"].clone()
        off[-1] = self.rows
        return off

    def backward(self, x, dy):
        """dy fp32 [T][N] -> gradients of the experts' weights and the router."""
        r = self.route
        rows = torch.zeros(self.rows + 1, self.N, dtype=torch.bfloat16, device=x.device)
        rows[self.at.reshape(-1)] = (self.w[..., None] * dy[:, None]).to(torch.bfloat16).reshape(-1, self.N)
        fp8g.fp8_quantize_transpose(rows[: self.rows], "e5m2", self.qa, self.sa)
        fp8g.fp8_quantize_transpose(self.xr, "e4m3", self.qb, self.sb)
        fp8g.grouped_gemm_fp8_wgrad(self.qa, "e5m2", self.sa, self.qb, "e4m3", self.sb, self.d_weight,
                                    group_offsets=r["group_offsets"])
        d_w = (self.picked * dy[:, None]).sum(2)
        d_logits = torch.empty_like(self.logits)
        if self.scored:
            fp8g.moe_route_scored_backward(self.logits, r["expert_ids"], d_w, self.one, r["counts"], r["routed"],
                                           d_logits, **self.scored)
        else:
            fp8g.moe_route_backward(self.logits, r["expert_ids"], d_w, self.one, r["counts"], r["routed"], d_logits,
                                    renormalise=True, loss_coef=self.balance)
        if self.adamw:
            self.d_router.copy_(d_logits.t() @ x.float())   # (the step's list holds its address)
        else:
            self.d_router = d_logits.t() @ x.float()
        return self.d_weight, self.d_router

    def step(self, x, target, lr, max_norm=1.0, mask=None):
        """One training step; the loss (a device tensor, balance included)."""
        y = self.forward(x, mask)
        err = y - target
        if mask is not None:
            err = err * mask[:, None]
        loss = err.square().mean() + self.route["loss"][0]
        grads = list(self.backward(x, 2.0 * err / err.numel()))
        fp8g.grad_norm_sq(grads, self.sumsq, self.clip_ws)
        if self.scored:
            counts = self.route["counts"].float()
            self.bias += 1e-3 * torch.sign(counts.mean() - counts)
        if self.adamw:
            self.steps += 1
            fp8g.adamw_step(self.tensors, self.steps, lr, sumsq=self.sumsq, max_norm=max_norm, norm=self.norm)
            return loss
        fp8g.grad_clip(grads, grads, self.sumsq, max_norm, self.norm)
        self.weight -= lr * grads[0].float()
        self.router -= lr * grads[1]
        return loss


def train(steps=30, tokens=1024, width=512, out=256, experts=8, top_k=2, lr=20.0, seed=0, **options):
    """Losses of `steps` steps."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    layer = MoELayer(tokens, width, out, experts, top_k, seed=seed, **options)
    teacher = torch.randn(out, width, device="cuda", generator=g) * width ** -0.5
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, device="cuda", generator=g).to(torch.bfloat16)
        losses.append(layer.step(x, x.float() @ teacher.t(), lr))
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--score", choices=["sigmoid", "softmax"])
    ap.add_argument("--adamw", type=int, choices=[32, 8], default=0, help="bits of the states")
    args = ap.parse_args()
    for i, v in enumerate(train(args.steps, lr=3e-3 if args.adamw else 20.0, score=args.score, adamw=args.adamw)):
        print(f"step {i:3d}  loss {v:.4f}", flush=True)
