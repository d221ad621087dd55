"""Definitions of the embedding, the dropout and the head's loss for the tests, in 64 bits, and how
far an output may be from them.

Tolerances count roundings: one to nearest is off by at most half a step, 2^-8 of the value in
bf16, 2^-11 in fp16, 2^-24 in fp32."""

import numpy as np
import torch

BF16, F16, F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
HALF = {torch.bfloat16: BF16, torch.float32: F32}


def bits(t):
    t = t.detach().cpu().contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).numpy()


def same_bits(a, b):
    return np.array_equal(bits(a), bits(b))


def rows_of(rows, dim, pitch, shift, dtype, scale, seed):
    """rows x dim inside rows of `pitch`, `shift` elements off the allocation's start; NaN between."""
    gen = torch.Generator().manual_seed(seed)
    buf = torch.full((rows * pitch + shift + 3,), float("nan"), dtype=dtype, device="cuda")
    t = buf[shift:shift + rows * pitch].view(rows, pitch)[:, :dim]
    t.copy_((scale * torch.randn(rows, dim, generator=gen)).to(dtype))
    return t


class Guarded:
    """rows x dim outputs inside rows of `pitch`, with a value around them that has to stay."""

    def __init__(self, rows, dim, pitch, shift, dtype, fill=7.0):
        self.fill = fill
        self.buf = torch.full((rows * pitch + shift + 5,), fill, dtype=dtype, device="cuda")
        self.t = self.buf[shift:shift + rows * pitch].view(rows, pitch)[:, :dim]

    def intact(self):
        kept = self.t.clone()
        self.t.fill_(self.fill)
        fine = bool((self.buf == self.fill).all())
        self.t.copy_(kept)
        return fine


# --- Philox 4 x 32 ----------------------------------------------------------------------------


def philox(counter, key, rounds=10):
    """counter: 4 arrays, key: 2 numbers; Salmon and others, 2011."""
    u = np.uint64
    c = [np.asarray(x, dtype=u) for x in counter]
    k = [int(x) for x in key]
    low = u(0xFFFFFFFF)
    for _ in range(rounds):
        p, q = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(q >> u(32)) ^ c[1] ^ u(k[0]), q & low, (p >> u(32)) ^ c[3] ^ u(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_bits(rows, dim, seed, offset, row0=0):
    """16 bits for each element of rows row0 on."""
    groups = -(-dim // 8)
    row = np.repeat(np.arange(row0, row0 + rows, dtype=np.uint64), groups)
    group = np.tile(np.arange(groups, dtype=np.uint64), rows)
    o = np.full(row.shape, 0, dtype=np.uint64)
    c = philox([group, row, o + np.uint64(offset & 0xFFFFFFFF), o + np.uint64(offset >> 32)],
               [seed & 0xFFFFFFFF, seed >> 32])
    halves = [h for w in c for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))]
    return np.stack(halves, 1).reshape(rows, groups * 8)[:, :dim]


def dropout(x, p, seed, offset, residual=None):
    """In fp32, operation by operation, rounded once to x's type: the same bits."""
    below = round(p * 65536)
    scale = np.float32(65536.0 / (65536 - below)) if below < 65536 else np.float32(0)
    keep = torch.from_numpy(dropout_bits(x.shape[0], x.shape[1], seed, offset) >= below)
    y = torch.where(keep, x.float().cpu() * float(scale), torch.zeros(()))
    if residual is not None:
        y = y + residual.float().cpu()
    return y.to(x.dtype)


# --- the embedding's gradient ------------------------------------------------------------------


def embedding_backward(tokens, dy, vocab, scale, old=None, padding=-1):
    """dweight and a bound of the fp32 sums' error, both 64 bits, on dy's device."""
    t = tokens.reshape(-1)
    keep = (t >= 0) & (t < vocab) & (t != padding)
    t, d = t[keep], dy[keep].double()
    zero = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device=dy.device)
    s = zero.clone().index_add_(0, t, d)
    size = zero.index_add_(0, t, d.abs())
    n = torch.bincount(t, minlength=vocab)[:, None]
    # n additions, the product with the scale, the scale's own rounding
    off = size * abs(scale) * (n + 3) * F32
    want = s * scale
    if old is not None:
        want = want + old.double()
        off = off + F32 * (want.abs() + off) * (n > 0)
    return want, off, n[:, 0]


# --- the head's loss ---------------------------------------------------------------------------


def loss(x, w, targets, scale=1.0, mean=True):
    """losses, loss, dhidden, dweight in 64 bits, and how far a kernel's may be off.

    A logit is a sum of `dim` products in fp32 (exact products of bf16 values; 2 roundings a term
    allow for an order and a width of the matrix instructions' own sums): off by z_off. A sum of
    exponentials: each off by its argument's roundings (of a logit's size, 4 of them) and the
    function's, a few; the sum of `vocab` terms by vocab / 64 (a tile's, then the tiles'). P is
    held in fp16, G in bf16, and G's products are summed in fp32 over the vocabulary or the rows."""
    t = targets.reshape(-1)
    vocab, dim = w.shape
    rows = torch.nonzero((t >= 0) & (t < vocab))[:, 0]
    X, W = x[rows].double(), w.double()
    z = X @ W.T.contiguous()
    zmax_off = 2 * dim * F32 * (X.abs() @ W.abs().T.contiguous()).amax(1, keepdim=True) if len(rows) else z[:, :1]
    at = torch.arange(len(rows), device=x.device)
    right = z[at, t[rows]]
    lse = torch.logsumexp(z, 1)
    others = z.clone()
    others[at, t[rows]] = -float("inf")
    ahead = torch.logsumexp(others, 1) - right            # log of sum exp(z_v - z_t)
    each = torch.where(ahead > 0, ahead + torch.log1p(torch.exp(-ahead)), torch.log1p(torch.exp(ahead)))
    # relative error of sum exp(z_v - z_t)
    rel = 2 * zmax_off[:, 0] + (4 * z.abs().amax(1) if vocab else 0) * F32 + (40 + vocab / 64 + vocab ** 0.5) * F32 if len(rows) else each
    each_off = rel * (1 - torch.exp(-each)) + 8 * F32 * each     # d loss = s / (1 + s) d log s
    losses = torch.zeros(len(t), dtype=torch.float64, device=x.device)
    losses_off = losses.clone()
    losses[rows], losses_off[rows] = each, each_off
    n = max(1, len(rows)) if mean else 1
    total, total_off = losses.sum() / n, losses_off.sum() / n + 2 * F32 * losses.sum() / n
    p = torch.exp(z - lse[:, None])
    g = p.clone()
    g[at, t[rows]] = torch.expm1(-each)
    g_off = g.abs() * (BF16 + F16 + BF16 * F16) + 2.0 ** -24 + p * (2 * rel + rel.square())[:, None]
    # P's subnormals in fp16: 2^-25 of a tile's largest exponential, which is at most 1 here
    k = scale / n
    dx = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    dx_off = dx.clone()
    dx[rows] = k * (g @ W)
    A = g.abs() + g_off
    dx_off[rows] = abs(k) * (g_off @ W.abs() + (2 * vocab + 4) * F32 * (A @ W.abs()))
    gt, at_ = g.T.contiguous(), A.T.contiguous()
    dw = k * (gt @ X)
    dw_off = abs(k) * (g_off.T.contiguous() @ X.abs() + (2 * len(rows) + 4) * F32 * (at_ @ X.abs()))
    return {"losses": (losses, losses_off), "loss": (total, total_off), "dhidden": (dx, dx_off), "dweight": (dw, dw_off)}


def near(got, want, off, half):
    """|got - want| <= off, and the output's own rounding of a value that may be that far off."""
    far = (got.double() - want).abs() - (off * (1 + half) + half * want.abs())
    return bool((far <= 0).all())
