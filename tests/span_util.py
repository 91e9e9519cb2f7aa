"""Batches for the tests of the attention of spans and behind shared prefixes."""
import numpy as np

from oracle import attention as A
from oracle import spans as S
from tests.test_gpu_attention import Case


class SpanCase(Case):
    """A Case with what its tokens see. groups: (sequences, shared tokens) of
    neighbouring sequences whose first pages are the same; None: span_attn."""

    def __init__(self, seed, ctx_lens, nds, kv, G, D, fmt, masked=False, groups=None, cap=0.0, slopes=None, window=0, first=None,
                 last=None, q_gain=3.0):
        super().__init__(seed, ctx_lens, nds, kv, G, D, fmt, masked=masked, q_gain=q_gain)
        self.groups = groups
        if groups is not None:
            at, self.cu_groups, self.shared = 0, [0], []
            for n, shared in groups:
                p = shared // 64
                for b in range(at, at + n):
                    self.table[b, :p] = self.table[at, :p]
                at += n
                self.cu_groups.append(at)
                self.shared.append(shared)
        if slopes is True:
            slopes = 2.0 ** (-8.0 * np.arange(1, self.H + 1) / self.H)
        as32 = lambda x, t: None if x is None else np.ascontiguousarray(x, t)  # noqa: E731
        self.mods = dict(cap=cap, window=window, slopes=as32(slopes, np.float32), first=as32(first, np.int32),
                         last=as32(last, np.int32))

    def place(self):
        """The place of each token."""
        return np.concatenate([np.arange(c, c + n) for c, n in zip(self.ctx, self.nds)] or [np.zeros(0)]).astype(np.int64)

    def workspace_size(self, ctx):
        if self.groups is None:
            return ctx.span_attn_workspace_size(self.Tq, self.B, self.H, self.kv, self.D)
        return ctx.shared_attn_workspace_size(self.Tq, self.B, len(self.shared), self.H, self.kv, self.D)

    def device(self):
        import torch
        super().device()
        for k in ("slopes", "first", "last"):
            self.d[k] = None if self.mods[k] is None else torch.from_numpy(self.mods[k]).cuda()
        if self.groups is not None:
            self.d["cu_groups"] = torch.tensor(self.cu_groups, dtype=torch.int32, device="cuda")
            self.d["shared"] = torch.tensor(self.shared, dtype=torch.int32, device="cuda")
        return self.d

    def run(self, ctx, out=None, lse=None, ws=None, q=None, stream=None, d=None):
        import torch
        d = self.device() if d is None else d
        q = d["q"] if q is None else q
        out = torch.full((self.Tq, self.H, self.D), 77.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        lse = torch.full((self.Tq, self.H), 77.0, device="cuda") if lse is None else lse
        if ws is None:
            # a workspace's old contents are scratch: NaN patterns must not matter
            ws = torch.full((self.workspace_size(ctx),), 0xFF, dtype=torch.uint8, device="cuda")
        args = (q, d["cache"], self.pages, self.fmt, self.kv, d["table"], d["lens"], d["cu"], out, ws)
        kw = dict(mask=d["mask"], lse=lse, scale=self.scale, cap=self.mods["cap"], window=self.mods["window"], slopes=d["slopes"],
                  first=d["first"], last=d["last"], stream=stream)
        if self.groups is None:
            ctx.span_attn(*args, **kw)
        else:
            ctx.shared_attn(*args, d["cu_groups"], d["shared"], **kw)
        return out, lse

    def reference(self):
        keys, vals = A.values(self.cache, self.pages, self.kv, self.D, self.fmt)
        return S.attend(self.q.astype(np.float64), self.kv, keys, vals, self.table, self.lens, self.cu, self.scale, self.mask,
                        self.mods["first"], self.mods["last"], self.mods["window"], self.mods["cap"], self.mods["slopes"])

    def check(self, out, lse, ref=None, rows=None):
        ref = self.reference() if ref is None else ref
        o, z = ref[:2]
        to, tl = S.tolerance(*ref, self.scale, self.D, float(self.lens.max()), self.mods["cap"])
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        rows = slice(None) if rows is None else rows
        fin = np.isfinite(z[rows])
        assert np.array_equal(gl[rows][~fin], z[rows][~fin])
        err = np.abs(gl[rows] - z[rows])
        assert np.all(err[fin] <= tl[rows][fin]), float(np.max((err / tl[rows])[fin]))
        err = np.abs(got[rows] - o[rows])
        assert np.all(err <= to[rows]), (float(np.max(err / to[rows])), np.argwhere(~(err <= to[rows]))[:5].tolist())
