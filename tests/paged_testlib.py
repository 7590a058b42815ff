"""A paged latent cache in plain float64, for the tests: batches of any shape, and what each paged call is defined
to compute. Errors are bounded element by element from the roundings that a call makes (derived at each bound)."""
import numpy as np
import torch

from mla_latent_kv_31_b200 import mla, synth

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}      # half a step, relative
NAN = float("nan")


def dims_of(dtype):
    return synth.V3 if dtype == "bf16" else synth.TINY


def handle(dtype):
    return mla.MLA(dims_of(dtype), None, mla.MLA_BF16 if dtype == "bf16" else mla.MLA_FP32)


class Case:
    """A batch with sequences of lens cached rows, the last tq of them new. Unowned pages and the rows behind each
    sequence hold NaN; table entries behind a sequence's last page are -7."""

    def __init__(self, dtype, page, lens, tq, seed=0, pad=0, spare=2, device="cuda", share=0):
        self.dtype, self.page, self.lens, self.tq, self.device = dtype, page, list(lens), list(tq), device
        self.dims = d = dims_of(dtype)
        self.W = d.d_c + d.d_r
        self.g = torch.Generator().manual_seed(seed)
        B, self.T, self.pad = len(self.lens), sum(self.tq), pad
        nb = [-(-n // page) for n in self.lens]
        self.num_pages = sum(nb) + spare
        order = torch.randperm(self.num_pages, generator=self.g).tolist()
        self.table = torch.full((B, max(max(nb), 1) + 1), -7, dtype=torch.int32)
        self.rows = []                                  # float64 rows of each sequence
        cache = torch.full((self.num_pages, page, self.W), NAN, dtype=torch.float64)
        at = 0
        for b, n in enumerate(self.lens):
            self.table[b, :nb[b]] = torch.tensor(order[at:at + nb[b]], dtype=torch.int32)
            at += nb[b]
            if share and b:                             # the first pages are sequence 0's
                k = min(share, self.lens[0] // page, (n - self.tq[b]) // page)
                self.table[b, :k] = self.table[0, :k]
            x = self.normal(n, self.W)
            pos = torch.arange(n)
            pages = self.table[b, pos // page].long()
            if share and b and k:
                x[:k * page] = self.rows[0][:k * page]
            cache[pages, pos % page] = x
            self.rows.append(x)
        self.cu = torch.tensor([0] + self.tq, dtype=torch.int64).cumsum(0)
        self.cache = cache.to(DT[dtype]).to(device)
        self.q = self.normal(self.T + pad, d.n_h, self.W)
        self.q[..., :d.d_c] *= 0.5
        self.q = self.q.to(DT[dtype]).double()
        self.d_table, self.d_cu = self.table.to(device), self.cu.to(device)
        self.d_lens = torch.tensor(self.lens, dtype=torch.int64, device=device)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, dtype=torch.float64).to(DT[self.dtype]).double()

    def on(self, x, dtype=None):
        return x.to(dtype or DT[self.dtype]).to(self.device).contiguous()

    @property
    def q_abs(self):
        return self.on(self.q[..., :self.dims.d_c])

    @property
    def q_rope(self):
        return self.on(self.q[..., self.dims.d_c:])

    def batch(self):
        return mla.PagedBatch(self.cache, self.d_table, self.d_cu, self.d_lens, self.T + self.pad)

    def tokens(self):
        """(token, sequence, position) of every new token."""
        return [(int(self.cu[b]) + k, b, n - t + k) for b, (n, t) in enumerate(zip(self.lens, self.tq)) for k in range(t)]

    def attend(self, t, rows):
        """(o, lse, A, bound of the scores' error) over the given rows. A = sum_j p_j |c_j|."""
        d = self.dims
        if rows.shape[0] == 0:
            return torch.zeros(d.n_h, d.d_c, dtype=torch.float64), torch.full((d.n_h,), -np.inf), None, None
        scale = (d.d_h + d.d_r) ** -0.5
        s = self.q[t] @ rows.T * scale
        p = torch.softmax(s, -1)
        # a score sums W products in fp32: each of at most W additions is off by 2^-23 (truncation allowed) of
        # the largest partial sum, itself at most sum |q||k|
        gamma = self.W * 2.0 ** -23 * scale * (self.q[t].abs() @ rows.abs().T).amax(-1)
        return p @ rows[:, :d.d_c], torch.logsumexp(s, -1), p @ rows[:, :d.d_c].abs(), gamma

    def check_attention(self, o, lse, rows_of):
        o, lse = o.double().cpu(), lse.double().cpu()
        for t, b, pos in self.tokens():
            rows = rows_of(t, b, pos)
            ro, rl, A, gamma = self.attend(t, rows)
            if A is None:
                assert torch.equal(o[t], ro) and torch.equal(lse[t], rl.double()), (t, b, pos)
                continue
            n = rows.shape[0]
            # weights: relative error 2 gamma (scores, through numerator and sum) and 2^-18 (exponentials); bf16
            # rounds each weight once more; fp32 sums of n terms; the output's own rounding
            rel = 2 * gamma + 2.0 ** -18 + n * 2.0 ** -23 + (HALF["bf16"] if self.dtype == "bf16" else 0.0)
            tol = rel[:, None] * A + HALF[self.dtype] * ro.abs() * (1 + rel[:, None])
            bad = (o[t] - ro).abs() - tol
            assert torch.isfinite(o[t]).all() and bad.max() <= 0, (t, b, pos, float(bad.max()))
            tol = gamma + 2.0 ** -18 + n * 2.0 ** -23 + 2.0 ** -23 * rl.abs()
            assert ((lse[t] - rl).abs() <= tol).all(), (t, b, pos, float((lse[t] - rl).abs().max()))

    # ---- summaries and selection
    def codes(self, x):
        """Codes and scale of rows x (float64 holding fp32 values), as the calls are defined."""
        x = x.float()
        s = x.abs().amax(-1, keepdim=True) / torch.tensor(127.0)
        ok = (s > 0) & torch.isfinite(s)
        c = torch.where(ok, x / torch.where(ok, s, 1.0), 0.0).round().clamp(-127, 127)
        return c.to(torch.int64), torch.where(ok, s, 0.0)

    def summaries(self, means):
        """Summary rows (uint8) of mean rows [n, W]."""
        c, s = self.codes(means)
        pitch = (self.W + 4 + 15) // 16 * 16
        out = torch.zeros(means.shape[0], pitch, dtype=torch.uint8)
        out[:, :self.W] = c.to(torch.int8).view(torch.uint8)
        out[:, self.W:self.W + 4] = s.float().contiguous().view(torch.uint8)
        return out

    def select(self, means, top_k, first, last):
        """Expected blocks of every new token from the pages' mean rows."""
        c, s = self.codes(means)
        qc, qs = self.codes(self.q)
        out = torch.full((self.T, top_k), -1, dtype=torch.int32)
        for t, b, pos in self.tokens():
            nb = pos // self.page + 1
            if nb <= top_k:
                out[t, :nb] = torch.arange(nb, dtype=torch.int32)
                continue
            pages = self.table[b, :nb].long()
            dots = (qc[t] @ c[pages].T).float()                       # exact: below 2^24
            score = (dots * qs[t]).amax(0) * s[pages, 0]
            order = sorted(range(first, nb - last), key=lambda g: (-float(score[g]), g))[:top_k - first - last]
            out[t] = torch.tensor(sorted([*range(first), *order, *range(nb - last, nb)]), dtype=torch.int32)
        return out


def rope(x, pos, dims):
    """Pairs (2m, 2m + 1) of the last axis turned by pos * theta_m (YaRN as the dims say), in float64."""
    d_r = dims.d_r
    m = torch.arange(d_r // 2, dtype=torch.float64)
    theta = dims.rope_base ** (-2.0 * m / d_r)
    mul = 1.0
    if getattr(dims, "yarn_s", 1.0) > 1.0:
        turns = dims.yarn_l0 * theta / (2 * np.pi)
        g = ((turns - dims.yarn_alpha) / (dims.yarn_beta - dims.yarn_alpha)).clamp(0, 1)
        theta = (1 - g) * theta / dims.yarn_s + g * theta
        mul = 0.1 * np.log(dims.yarn_s) + 1.0
    a = pos * theta
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * a.cos() - x1 * a.sin(), x0 * a.sin() + x1 * a.cos()], -1).flatten(-2) * mul
