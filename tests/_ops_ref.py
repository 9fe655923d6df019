"""64-bit references of the operators of include/moe_ops.h, and the inputs and
error bounds their tests share.

Bounds count roundings.  U32 = 2^-24 is half a step of fp32 relative to the
value; sums on the tensor cores may drop the bits below their result instead of
rounding them, a whole step, 2 U32, per addition.  A rounding to bf16 is off by
at most 2^-8 of the value and one to e4m3 by 2^-4 (below 2^-6, by 2^-10)."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
BF16 = 2.0 ** -8
E4M3 = 2.0 ** -4
BLOCK = 128


def nb(n: int) -> int:
    return -(-n // BLOCK)


def gen(seed: int, device="cuda") -> torch.Generator:
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def spread(s, rows, cols):
    """Block scales [..., R, C] over [..., rows, cols], 64 bits."""
    r = torch.arange(rows, device=s.device) // BLOCK
    c = torch.arange(cols, device=s.device) // BLOCK
    return s.double()[..., r, :][..., c]


def weights64(codes, scales):
    return codes.view(torch.float8_e4m3fn).double() * spread(scales, codes.shape[-2],
                                                             codes.shape[-1])


def rows64(codes, scales):
    c = torch.arange(codes.shape[1], device=codes.device) // BLOCK
    return codes.view(torch.float8_e4m3fn).double() * scales.double()[:, c]


def quant_rows(x):
    """Rows to (codes, scales), as a caller's own quantiser would."""
    T, d = x.shape
    p = torch.zeros(T, nb(d) * BLOCK, device=x.device)
    p[:, :d] = x.float()
    p = p.view(T, nb(d), BLOCK)
    s = p.abs().amax(2) / 448.0
    q = torch.where(s[:, :, None] > 0, p / s[:, :, None], p).view(T, -1)[:, :d]
    return q.to(torch.float8_e4m3fn).contiguous(), s.contiguous()


def rand_weights(shape, seed, std=0.05):
    """(codes, scales) of N(0, std) weights [..., R, C] with uneven scales."""
    g = gen(seed)
    q = (torch.randn(shape, device="cuda", generator=g) * (448 / 4.2)).clamp(-448, 448)
    s = torch.rand(*shape[:-2], nb(shape[-2]), nb(shape[-1]), device="cuda", generator=g) + 0.5
    return q.to(torch.float8_e4m3fn), s * (std * 4.2 / 448)


# ------------------------------------------------------------------- norms
def norm64(x, y, gate, kind, pre_w, post_w, post, sigmoid, centred, a, b, eps):
    """(r, h, bound on the fp32 error of r, the same of h), 64 bits."""
    off = 1.0 if centred else 0.0
    one = torch.ones((), dtype=torch.float64, device=x.device)
    W = lambda w: one if w is None else w.double() + off   # noqa: E731
    x = x.double()
    r, mag = a * x, (a * x).abs()
    if y is not None:
        u = y.double()
        if post:
            u = u * (u.pow(2).mean(1, keepdim=True) + eps).rsqrt() * W(post_w)
        if kind != "none":
            g = gate.double()
            g = torch.sigmoid(g) if sigmoid else g
            u = u * (g[:, None] if kind == "token" else g)
        r = r + b * u
        mag = mag + (b * u).abs()
    inv = (r.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    h = r * inv * W(pre_w)
    # roundings on the way to r: two squares' sums (at most 32 additions deep,
    # halved by the root), rsqrt, exp and division 2 steps each, and 8 products
    # or sums: below 64 half steps of the terms.  h adds the same again.
    dr = 64 * U32 * mag
    dh = (64 * U32 * h.abs()) + dr * inv * W(pre_w).abs()
    # a common relative error of the row's mean square from dr
    drel = (dr.pow(2).mean(1, keepdim=True)).sqrt() * inv
    return r, h, dr, dh + h.abs() * drel


# ---------------------------------------------------------------- products
def product64(a, sa, w, sw):
    """(c, bound without the bf16 rounding) of one product, 64 bits."""
    A, W = rows64(a, sa), weights64(w, sw)
    c = A @ W.T
    # 128 products of a block and ceil(K/128) blocks are added, each addition
    # off by at most a whole fp32 step of a partial sum that is below S; the
    # scale product and its use round twice more
    S = A.abs() @ W.abs().T
    return c, (BLOCK + nb(a.shape[1]) + 2) * 2 * U32 * S


# ------------------------------------------------------------------- layer
class Layer64:
    """Random layer with e4m3 experts and its 64-bit reference."""

    def __init__(self, d, E, k, F, Fs, seed, bias=True, router_std=0.02):
        from routed_expert_ffn_06_b200 import moe_ops
        g = gen(seed)
        self.d, self.E, self.k, self.F, self.Fs = d, E, k, F, Fs
        self.router_w = torch.randn(E, d, device="cuda", generator=g) * router_std
        self.bias = torch.randn(E, device="cuda", generator=g) * 0.5 if bias else None
        self.gu, self.gus = rand_weights((E, 2, F, d), seed + 1)
        self.dn, self.dns = rand_weights((E, d, F), seed + 2)
        self.sgu = self.sgus = self.sdn = self.sdns = None
        if Fs:
            self.sgu, self.sgus = rand_weights((2, Fs, d), seed + 3)
            self.sdn, self.sdns = rand_weights((d, Fs), seed + 4)
        self.handle = moe_ops.make_fp8_layer(k, self.router_w, self.bias, self.gu, self.gus,
                                             self.dn, self.dns, self.sgu, self.sgus, self.sdn,
                                             self.sdns)

    def run(self, x, ws=None):
        from routed_expert_ffn_06_b200 import moe_ops
        T = x.shape[0]
        ws = moe_ops.alloc_fp8_workspace(self.handle, max(T, 1)) if ws is None else ws
        y = torch.full_like(x, float("nan"))
        ids = torch.full((T, self.k), -1, dtype=torch.int32, device="cuda")
        w = torch.full((T, self.k), float("nan"), device="cuda")
        moe_ops.moe_fp8_layer_forward(self.handle, x, T, y, ws, ids, w)
        return y, ids, w, ws

    def logits64(self, x):
        """(logits, bound of their fp32 error)."""
        W = self.router_w.double()
        l = x.double() @ W.T
        S = x.double().abs() @ W.abs().T
        if self.bias is not None:
            l, S = l + self.bias.double(), S + self.bias.double().abs()
        return l, (self.d + 8) * U32 * S

    def _ffn(self, x, gu, gus, dn, dns, mix):
        """One expert's weighted output and its error bound for all rows of x;
        mix: the rows' weights [T, 1]."""
        Wg, Wu, Wd = weights64(gu[0], gus[0]), weights64(gu[1], gus[1]), weights64(dn, dns)
        gam = (BLOCK + 2 * nb(self.d) + 4) * 2 * U32
        g, u = x @ Wg.T, x @ Wu.T
        dg, du = gam * (x.abs() @ Wg.abs().T), gam * (x.abs() @ Wu.abs().T)
        s = g * torch.sigmoid(g)
        h = s * u * mix
        # |silu'| <= 1.1; exp, division and products are off by less than 16 half
        # steps; the down product takes h in fp16 (half a step is 2^-11 of the
        # value) after a scale that leaves at most 2^-39 of the token's largest h
        # below; the tokens' two e4m3 terms leave 2^-21 of the largest of each 128
        # columns, here of the whole row, next to every weight
        top = x.abs().amax(1, keepdim=True) * 2.0 ** -21
        dg = dg + top * Wg.abs().sum(1)
        du = du + top * Wu.abs().sum(1)
        dh = ((1.1 * dg * (u.abs() + du) + s.abs() * du) * mix + (2.0 ** -11 + 16 * U32) * h.abs()
              + 2.0 ** -39 * h.abs().amax(1, keepdim=True))
        items = nb(Wd.shape[1])
        gam2 = (2 * BLOCK + items + 4) * 2 * U32
        return h @ Wd.T, dh @ Wd.abs().T + gam2 * (h.abs() @ Wd.abs().T), h.abs() @ Wd.abs().T

    def check(self, x, y, ids, w):
        """The routing and outputs of every token against the reference."""
        T = x.shape[0]
        l, dl = self.logits64(x)
        ids = ids.long()
        assert ((ids >= 0) & (ids < self.E)).all()
        assert all(len(set(r)) == self.k for r in ids.tolist()), "an expert twice"
        sel, dsel = l.gather(1, ids), dl.gather(1, ids)
        assert ((sel[:, :-1] - sel[:, 1:]) >= -(dsel[:, :-1] + dsel[:, 1:])).all(), "order"
        rest = l.scatter(1, ids, float("-inf"))
        assert (rest.amax(1) <= sel[:, -1] + dsel[:, -1] + dl.amax(1)).all(), "selection"
        w64 = torch.softmax(sel, 1)
        # a logit error e moves a weight by at most w (exp(2 e) - 1)
        dw = w64 * (torch.expm1(2 * dsel.amax(1, keepdim=True)) + 32 * U32)
        assert ((w.double() - w64).abs() <= dw).all(), "weights"
        xd = x.double()
        out = torch.zeros(T, self.d, dtype=torch.float64, device="cuda")
        bound, size = torch.zeros_like(out), torch.zeros_like(out)
        for e in sorted(set(ids.flatten().tolist())):
            mix = torch.where(ids == e, w.double(), torch.zeros_like(w64)).sum(1, keepdim=True)
            o, b, s = self._ffn(xd, self.gu[e], self.gus[e], self.dn[e], self.dns[e], mix)
            out, bound, size = out + o, bound + b, size + s
        if self.Fs:
            o, b, s = self._ffn(xd, self.sgu, self.sgus, self.sdn, self.sdns,
                                torch.ones(T, 1, dtype=torch.float64, device="cuda"))
            out, bound, size = out + o, bound + b, size + s
        # the experts' parts are added in at most (T k + 1) ceil(F/128) + 16 steps
        steps = (8 * self.k + 1) * nb(max(self.F, self.Fs)) + 16
        bound = bound + steps * U32 * size
        err = (y.double() - out).abs()
        tol = bound * (1 + BF16) + BF16 * out.abs()
        assert (err <= tol).all(), f"worst {(err / tol.clamp_min(1e-300)).max().item():.3f} of the bound"
