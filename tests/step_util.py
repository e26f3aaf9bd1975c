"""Plain 64-bit forms of the step's operators (page tables and slots, cache
writes, tree attention, packed prompts) and the bound their results are held
to.

Bound of an attention output, element by element, with w the exact weights
(sum 1), A = sum_t w_t |v_t| and L the tokens seen:
  * each weight is rounded to fp16 before it multiplies V: relative 2^-11 (half
    a step), or, below the smallest normal fp16, absolute 2^-25 against an
    exp-sum of at least 1 (the reference maximum is never above the row's):
    at most 2^-11 A + L 2^-25 max|v|;
  * the score is an fp32 sum of D exact products: with truncation at every
    step off by at most D 2^-23 sum_d |q_d k_d| scale, which for the N(0, 1)
    values here (sum_d |q_d k_d| < D) is below D^2 scale 2^-23, so the weights (numerator and exp-sum) are off by at most twice that,
    relatively; the exponential itself (2^-22), its argument's rounding
    (|score| log2(e) < 2^5: 2^-19) and the fp32 sums of L positive terms
    (L 2^-24 with sequential adds) come on top;
  * an fp16 result is rounded once more: 2^-11 |out|.
"""
import numpy as np
import torch


def attention(q, k, v, seen, scale):
    """softmax(q k^T scale) v over ``seen``: q [n, H, D], k, v [L, Hkv, D] (any
    float type), seen bool [n, L].  Returns (out, A), float64 [n, H, D]; a row
    that sees nothing is zero."""
    dev = q.device
    q, k, v = (x.detach().double() for x in (q, k, v))
    seen = torch.as_tensor(seen, device=dev)
    n, H, D = q.shape
    G = H // k.shape[1]
    out = torch.zeros((n, H, D), dtype=torch.float64, device=dev)
    A = torch.zeros_like(out)
    empty = ~seen.any(1)
    for h in range(H):
        z = (q[:, h] @ k[:, h // G].T * scale).masked_fill(~seen, -torch.inf)
        w = torch.exp(z - z.amax(1, keepdim=True).masked_fill(empty[:, None], 0.0))
        w = w / w.sum(1, keepdim=True).masked_fill(empty[:, None], 1.0)
        out[:, h] = w @ v[:, h // G]
        A[:, h] = w @ v[:, h // G].abs()
    return out.cpu().numpy(), A.cpu().numpy()


def bound(out, A, L, D, vmax, half, scale=None):
    scale = D ** -0.5 if scale is None else abs(scale)
    weights = 2.0 ** -11 + 2 * (D * D * scale * 2.0 ** -23 + 2.0 ** -19 + 2.0 ** -22 + L * 2.0 ** -24)
    tol = weights * A + L * 2.0 ** -25 * vmax
    if half:
        tol = tol + 2.0 ** -11 * (np.abs(out) + tol) + 2.0 ** -25
    return tol + 1e-7


def assert_attention(got, ref, A, L, D, vmax, what="", scale=None):
    half = got.dtype == torch.float16
    g = got.detach().cpu().numpy().astype(np.float64)
    assert g.shape == ref.shape, (g.shape, ref.shape)
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    over = np.abs(g - ref) / bound(ref, A, L, D, vmax, half, scale)
    worst = over.max() if over.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} times the bound"
    return worst


def tree_seen(parents, context):
    """seen [n, context + n] of a tree's rows: the context, ancestors, itself."""
    n = len(parents)
    seen = np.zeros((n, context + n), dtype=bool)
    seen[:, :context] = True
    for i, p in enumerate(parents):
        j = i
        while j >= 0:
            seen[i, context + j] = True
            p = parents[j]
            j = p if 0 <= p < j else -1
    return seen


def slots(context, query, tables, free, start, block_size, num_rows):
    """The plain form of paged_kv_slots for counts that are in order: (slots,
    positions, cu, lens, end, tables)."""
    tables = np.array(tables)
    S = len(context)
    slot = np.full(num_rows, -1, dtype=np.int64)
    position = np.full(num_rows, -1, dtype=np.int64)
    cu, lens, at = [0], [], int(start)
    for s in range(S):
        c, n = int(context[s]), int(query[s])
        owned = -(-c // block_size)
        for j in range(owned, -(-(c + n) // block_size)):
            tables[s, j] = free[at]
            at += 1
        for i in range(n):
            t = c + i
            position[cu[-1] + i] = t
            slot[cu[-1] + i] = tables[s, t // block_size] * block_size + t % block_size
        cu.append(cu[-1] + n)
        lens.append(c + n)
    return slot, position, np.array(cu), np.array(lens, dtype=np.int64), at, tables


def packed_seen(n):
    return np.tril(np.ones((n, n), dtype=bool))
