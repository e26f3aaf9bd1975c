"""Plain 64-bit forms of the rotary write and of attention over latent vectors, and
the bounds their results are held to.

Rotation: the kernel's place on the circle is off by 2^-32 of a turn (the fraction's
low bits) and, as an fp32 number of half turns, by 2^-25 of itself: 1.1e-7 radians in
all; sine and cosine by 2 ulp, 2^-22 at most near 1.  So each of them is within 2^-21;
the two products and their difference round three times (2^-24 of |a| + |b| each), the
magnitude's product once more: together below 2^-20 m (|a| + |b|); then the result is
rounded to fp16, 2^-11 of itself or 2^-25.

Attention: the bound of step_util with D = the width of a score's sum; its weights and
output are held the same way.
"""
import numpy as np
import torch

from step_util import bound


def turned(x, positions, inv_freq, interleaved, magnitude=1.0):
    """x [rows, heads, D] with the first 2 len(inv_freq) values turned: (result, bound)."""
    x = x.detach().double()
    m = inv_freq.numel()
    angle = positions.double()[:, None, None] * inv_freq.double()
    c, s = angle.cos() * magnitude, angle.sin() * magnitude
    i = torch.arange(m, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + m)
    a, b = x[..., first], x[..., second]
    y, tol = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    near = 2.0 ** -20 * abs(magnitude) * (a.abs() + b.abs())
    tol[..., first] = near + 2.0 ** -11 * (y[..., first].abs() + near) + 2.0 ** -25
    tol[..., second] = near + 2.0 ** -11 * (y[..., second].abs() + near) + 2.0 ** -25
    return y, tol


def assert_turned(got, ref, tol, what=""):
    off = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    over = (off > tol).nonzero()
    assert over.numel() == 0, (f"{what}: {over.shape[0]} values past the bound, first "
                               f"{over[0].tolist()}: {off[tuple(over[0])]} > {tol[tuple(over[0])]}")


def attention(q, k, v, seen, scale):
    """softmax(q k^T scale) v: q [n, H, W], k [L, H or 1, W], v [L, H or 1, D], seen bool
    [n, L].  Returns (out, A) float64 [n, H, D], A the weighted sum of |v|; a row that
    sees nothing is zero."""
    dev = q.device
    q, k, v = (x.detach().double() for x in (q, k, v))
    seen = torch.as_tensor(seen, device=dev)
    n, H = q.shape[:2]
    out = torch.zeros((n, H, v.shape[2]), dtype=torch.float64, device=dev)
    A = torch.zeros_like(out)
    empty = ~seen.any(1)
    for h in range(H):
        kh, vh = (x[:, h if x.shape[1] > 1 else 0] for x in (k, v))
        z = (q[:, h] @ kh.T * scale).masked_fill(~seen, -torch.inf)
        w = torch.exp(z - z.amax(1, keepdim=True).masked_fill(empty[:, None], 0.0))
        w = w / w.sum(1, keepdim=True).masked_fill(empty[:, None], 1.0)
        out[:, h] = w @ vh
        A[:, h] = w @ vh.abs()
    return out.cpu().numpy(), A.cpu().numpy()


def assert_attention(got, ref, A, L, width, vmax, scale, what=""):
    g = got.detach().cpu().numpy().astype(np.float64)
    assert g.shape == ref.shape, (g.shape, ref.shape)
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    over = np.abs(g - ref) / bound(ref, A, L, width, vmax, got.dtype == torch.float16, scale)
    worst = over.max() if over.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} times the bound"
    return worst


class LatentCase:
    """Requests over a latent cache: shuffled pages, other requests' pages behind a
    table's end, NaN in every cached row that belongs to none."""

    def __init__(self, lens, new, H, R=512, P=64, BS=16, seed=0, dev="cuda:0", q="packed",
                 pad_token=0, pad_page=0):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.lens, self.new, self.H, self.R, self.P, self.BS, self.dev = lens, new, H, R, P, BS, dev
        pages = [-(-n // BS) for n in lens]
        total = sum(pages) + 3
        at = np.concatenate([[0], np.cumsum(pages)]).astype(int)
        ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        MB = max([1] + pages)
        entry = torch.arange(MB)[None, :] + torch.as_tensor(at[:-1])[:, None]
        self.tables = ids[(entry % total).to(dev)].contiguous()
        self.NB = total
        W = R + P
        buf = torch.full((total, BS + pad_page, W + pad_token), float("nan"), dtype=torch.float16,
                         device=dev)
        self.cache = buf[:, :BS, :W]
        self.rows = []
        for s, n in enumerate(lens):
            x = torch.randn((n, W), generator=g, device=dev).half()
            self.rows.append(x)
            for j in range(pages[s]):
                part = x[j * BS:(j + 1) * BS]
                self.cache[int(self.tables[s, j]), :part.shape[0]] = part
        self.cu = torch.as_tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=dev)
        self.T = int(sum(new))
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        if q == "packed":          # parts of one tensor
            both = torch.randn((self.T, H, W), generator=g, device=dev).half()
            self.q, self.q_rope = both[..., :R], both[..., R:]
        else:                      # a batched product's output, and a tensor of its own
            self.q = torch.randn((H, self.T, R), generator=g, device=dev).half().transpose(0, 1)
            self.q_rope = torch.randn((self.T, H, P), generator=g, device=dev).half()
        self.scale = (128 + P) ** -0.5

    def run(self, dtype=torch.float16, single=False, max_q=None, extra_rows=0, **kw):
        import paged_gqa_decode_03_gb300 as pgd
        out = torch.full((self.T, self.H, self.R), float("nan"), dtype=dtype, device=self.dev)
        pgd.paged_latent_attention(out, self.q, self.q_rope, self.cache, self.tables, self.seq_lens,
                                   self.scale, cu_seqlens_q=None if single else self.cu,
                                   max_q_len=max(self.new) if max_q is None else max_q, **kw)
        torch.cuda.synchronize()
        return out

    def expected(self, s, scale=None):
        n, L = self.new[s], self.lens[s]
        r0 = int(sum(self.new[:s]))
        seen = np.arange(L)[None, :] <= (L - n + np.arange(n))[:, None]
        q = torch.cat([self.q[r0:r0 + n], self.q_rope[r0:r0 + n]], -1)
        k = self.rows[s][:, None]
        ref, A = attention(q, k, k[..., :self.R], seen, self.scale if scale is None else scale)
        return slice(r0, r0 + n), ref, A

    def check(self, out, what="", seqs=None):
        for s in range(len(self.lens)) if seqs is None else seqs:
            if self.new[s] == 0:
                continue
            rows, ref, A = self.expected(s)
            vmax = float(self.rows[s].abs().max()) if self.lens[s] else 0.0
            assert_attention(out[rows], ref, A, self.lens[s], self.R + self.P, vmax, self.scale,
                             f"{what} seq {s}")
