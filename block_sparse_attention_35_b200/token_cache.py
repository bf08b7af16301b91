"""A bounded 4-bit cache of single tokens: attend, account, evict (include/pbsa.h, token cache).

Beside ``SparseForcingAttention``, whose caches hold blocks of video tokens in bf16, this one
holds tokens one by one, for streams that are generated token by token or in small steps.  The
object owns the device tensors; every step of the method runs in the kernels behind
``pbsa.pbsa_kv4_*``.

    cache = TokenCache(B, Hq, Hkv, D, capacity=4096, n_sink=4, n_recent=256)
    out = cache.step(q, k, v)        # rows for the new tokens, append, causal attention

Until the cache is full the new tokens take empty rows; then a step of T tokens takes the T rows
that drew the least attention so far, sparing the sequence's first ``n_sink`` and its last
``n_recent`` tokens.  A padded sequence, with fewer tokens than T, takes what is empty first and
then the first of those T rows in the order of the cache, not the lightest of them.
Nothing in a step waits for the GPU, and a step can be captured into a CUDA graph.  A step's output
is a buffer that the next step of the same T writes again.  The buffers of the last ``_KEEP``
lengths are kept for the next step of their length, and those of a captured step as long as the
cache."""
from __future__ import annotations

import torch

from . import pbsa as P


_KEEP = 4


class TokenCache:
    def __init__(self, B: int, Hq: int, Hkv: int, D: int, capacity: int, dtype=torch.bfloat16,
                 n_sink: int = 4, n_recent: int = 64, k_unit: float = 1.0, v_unit: float = 1.0,
                 device="cuda"):
        self.cfg = P.make_kv4_config(B, Hq, Hkv, D, capacity, dtype, k_unit, v_unit)
        P.pbsa_validate_kv4_config(self.cfg)
        if n_sink < 0 or n_recent < 0:
            raise ValueError("n_sink and n_recent must be >= 0")
        self.B, self.Hq, self.Hkv, self.D, self.capacity = B, Hq, Hkv, D, capacity
        self.dtype, self.n_sink, self.n_recent = dtype, n_sink, n_recent
        dev = self.device = torch.device(device)
        u8 = dict(dtype=torch.uint8, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        rows = (B, Hkv, capacity)
        self.k_codes = torch.zeros(*rows, D // 2, **u8)
        self.k_scales = torch.zeros(*rows, D // 16, **u8)
        self.v_codes = torch.zeros(*rows, D // 2, **u8)
        self.v_scales = torch.zeros(*rows, D // 16, **u8)
        self.pos = torch.full(rows, -1, **i32)
        self.mass = torch.zeros(*rows, dtype=torch.float32, device=dev)
        self.cache = P.make_kv4_cache(self.cfg, self.k_codes, self.k_scales, self.v_codes,
                                      self.v_scales, self.pos)
        self.device = self.pos.device
        self.seen = torch.zeros(B, **i32)       # tokens of every sequence so far
        self.kv_len = torch.zeros(B, **i32)     # rows in use
        self.status = torch.zeros(1, **i32)
        self._count = torch.arange(capacity, **i32)
        self._turn = torch.arange(capacity, device=dev) - capacity
        self._steps = {}                        # by T: see _buffers
        self._most = 0   # rows in use, at most; None: a replayed step adds to them unseen

    def _buffers(self, T: int):
        """The tensors of a step of T tokens, allocated on its first use; the least recently used
        ones are given up, but for those whose addresses a graph holds."""
        s = self._steps.pop(T, None)
        capturing = torch.cuda.is_current_stream_capturing()
        if s is None:
            if not capturing:
                spare = [n for n, x in self._steps.items() if not x["captured"]]
                for n in spare[:max(0, len(spare) + 1 - _KEEP)]:
                    for t in self._steps.pop(n).values():
                        if torch.is_tensor(t):   # this stream may still work on it
                            t.record_stream(torch.cuda.current_stream(self.device))
            dev = self.device
            s = dict(
                captured=False,
                ar=self._count[:T],
                rows=torch.empty(self.B, self.Hkv, T, dtype=torch.int32, device=dev),
                out=torch.empty(self.B, T, self.Hq, self.D, dtype=self.dtype, device=dev),
                lse=torch.empty(self.B, self.Hq, T, dtype=torch.float32, device=dev),
                ws=torch.empty(P.pbsa_kv4_workspace_size(self.cfg, T), dtype=torch.uint8,
                               device=dev))
        if capturing:
            s["captured"], self._most = True, None
        self._steps[T] = s   # the last: in order of use
        return s

    def step(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_new=None):
        """T new tokens of every sequence (n_new [B] int32 on the device: how many of them are
        tokens, from 0 to T, beyond which it counts as the nearer of the two; the rest is padding;
        None: all) enter the cache and attend to it and to each other causally.  q [B, T, Hq, D],
        k, v [B, T, Hkv, D], normalised and rotated already.  Returns the output [B, T, Hq, D]
        (zeros for padding), which the next step of T tokens writes again.  What does not fit is
        refused before anything changes."""
        T = q.shape[1]
        for name, t, H in (("q", q, self.Hq), ("k", k, self.Hkv), ("v", v, self.Hkv)):
            P._want_heads(t, name, (self.B, T, H, self.D), self.dtype, self.device)
        if n_new is not None and (n_new.shape != (self.B,) or n_new.dtype not in (torch.int32, torch.int64)
                                  or n_new.device != self.device):
            raise ValueError(f"n_new is not a tensor of {self.B} int32 on {self.device}")
        if T + self.n_sink + self.n_recent > self.capacity:
            raise ValueError(f"a step of {T} tokens does not fit beside {self.n_sink} sink and "
                             f"{self.n_recent} recent tokens in {self.capacity} rows")
        s = self._buffers(T)
        pos = self.seen[:, None] + s["ar"]
        n = T
        if n_new is not None:
            n = n_new.clamp(0, T).int()
            pos = torch.where(s["ar"] < n[:, None], pos, -1)
        P.pbsa_kv4_evict(self.cfg, self.pos, self.mass, self.n_sink, self.seen - self.n_recent,
                         s["rows"], self.status)
        rows = s["rows"]
        if n_new is not None and T > 1 and (self._most is None or self._most + T > self.capacity):
            # Empty rows first, where rows in use may be among the chosen.  Those in use are the
            # first kv_len, so that of the T chosen ones, in row order, the last capacity - kv_len
            # are empty: they are turned to the front.
            turn = (self._turn[:T] + self.kv_len.clamp(min=self.capacity - T)[:, None]) % T
            rows = rows.gather(2, turn[:, None].expand(rows.shape))
        P.pbsa_kv4_append(self.cfg, self.cache, k, v, pos, rows, self.mass, self.status)
        if self._most is not None:
            self._most = min(self._most + T, self.capacity)
        self.seen += n
        torch.clamp(self.seen, max=self.capacity, out=self.kv_len)
        P.pbsa_kv4_attn(self.cfg, self.cache, q, pos, self.kv_len, s["out"], s["lse"], self.mass,
                        s["ws"], self.status)
        return s["out"]
