"""The 4-bit paged KV cache in plain 64-bit arithmetic on the CPU, and batches to test it with."""
import math

import torch

Q = {4: (math.sqrt(7.0), -8, 7), 3: (3.0, -4, 3), 8: (127.0, -128, 127)}
U = 2.0 ** -24  # half a step of fp32


def quantise(x, bits, eps=1e-5):
    """(codes, step) of rows x in 64 bits."""
    x = x.double()
    q, lo, hi = Q[bits]
    scale = (x.abs().mean(-1) if bits == 4 else x.abs().amax(-1)) + float(torch.tensor(eps, dtype=torch.float32))
    return (x * (q / scale)[..., None]).round().clamp(lo, hi).to(torch.int64), scale / q


class Batch:
    """A ragged batch on the CPU: lens, new rows per sequence, pages in a shuffled order; before and behind the
    sequences' rows lie `lead` and `tail` rows of nobody."""

    def __init__(self, lens, new, page, seed=0, lead=0, tail=0, spare=2, first_page=0, width=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.page = list(lens), list(new), page
        need = [-(-m // page) for m in lens]
        self.pages = first_page + sum(need) + spare
        order = (torch.randperm(sum(need) + spare, generator=g) + first_page).tolist()
        self.width = max(need + [1]) if width is None else width
        self.table = torch.full((len(lens), self.width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.starts = torch.tensor([lead] + [lead + sum(new[:i + 1]) for i in range(len(new))], dtype=torch.int32)
        self.rows = lead + sum(new) + tail

    def tensors(self, device):
        return (self.table.to(device), torch.tensor(self.lens, dtype=torch.int32, device=device), self.starts.to(device))

    def places(self):
        """(row, sequence, position, page, offset) of every row with a position."""
        for b, (m, n) in enumerate(zip(self.lens, self.new)):
            for i in range(n):
                pos = m - n + i
                if pos >= 0:
                    yield int(self.starts[b]) + i, b, pos, int(self.table[b, pos // self.page]), pos % self.page


def values(codes, step, bos, batch, b):
    """All cached values of sequence b as [length, heads, dim] in 64 bits, from CPU copies of one side's tensors."""
    m = batch.lens[b]
    pos = torch.arange(m)
    at, off = batch.table[b].long()[pos // batch.page], pos % batch.page
    held = codes[at, :, off].long()
    x = torch.stack((((held & 15) ^ 8) - 8, ((held >> 4) ^ 8) - 8), -1).flatten(-2).double()
    if m:
        x[0] = bos[at[0]].double()
    return x * step[at, :, off].double()[..., None]


def attention(q, k, v, scale, causal, window):
    """q [n, Hq, D] at the last n of the positions of k, v [m, H, D]: (out, lse, bound on |s|, sum of p |v|)."""
    n, heads, _ = q.shape
    m, kv, _ = k.shape
    group = heads // kv
    q, k, v = q.double(), k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    z = torch.einsum("nhd,mhd->hnm", q, k) * scale
    size = torch.einsum("nhd,mhd->hnm", q.abs(), k.abs()) * abs(scale)
    p, t = torch.arange(m - n, m)[:, None], torch.arange(m)
    hide = torch.zeros((n, m), dtype=torch.bool)
    if causal:
        hide |= t > p
        if window:
            hide |= t <= p - window
    z = z.masked_fill(hide, -math.inf)
    size = size.masked_fill(hide, 0.0)
    lse = torch.logsumexp(z, -1) if m else torch.full((heads, n), -math.inf, dtype=torch.float64)
    w = torch.exp(z - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
    out = torch.einsum("hnm,mhd->nhd", w, v)
    mass = torch.einsum("hnm,mhd->nhd", w, v.abs())
    top = size.amax(-1) if m else torch.zeros((heads, n), dtype=torch.float64)
    return out, lse.T, top.T, mass


def attention_bounds(out, top, mass, dim, length, dtype, largest):
    """How far out and lse may be off.  A score is a sum of dim products in fp32 and some scalings: its error is a
    sum of about dim + 8 independent roundings of at most 2 U (the tensor cores cut where they add) relative to
    sum |q k|, taken at 2 sqrt(dim) + 8 times 2 U.  A weight's relative error is that of its score (twice: once in
    the numerator, once in the sum) and some roundings of the exponential; the sums over positions add
    2 sqrt(length) roundings.  bf16 calls round weights to fp16 (2^-11) and the output to bf16 (2^-8).

    Weights far below the row's largest reach the end of fp16's range.  Weights w step / 2^e, with 2^e at most the
    largest step so far, are held as multiples of 2^-24 where the largest w is at least 2^3 (bf16 calls) or
    2^13 (fp32 calls, in their second part): each is off by at most 2^-25, so that of the largest by 2^-28 (2^-38),
    times 2^e and a code of at most 8 (127 at position 0).  A row with the step 2^e has a code of 1 or
    more, so 2^e is at most the largest |value| of the sequence (`largest`)."""
    score = 2 * U * (2 * math.sqrt(dim) + 8) * top
    rel = 2 * score + (2 * math.sqrt(length) + 32) * U
    if dtype == torch.bfloat16:
        rel = rel + 2.0 ** -11
    err = rel[..., None] * mass + out.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else U) + 1e-37
    err = err + (2.0 ** -28 if dtype == torch.bfloat16 else 2.0 ** -38) * (8 * length + 127) * largest
    return err, score + (2 * math.sqrt(length) + 32) * U
