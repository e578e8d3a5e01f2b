"""Plain definitions of the key and value cache in 64 bits, and a cache on the device to check against them.

`Cache` keeps pages in the layout asked for ("head": a page's tokens of one head together; "token": a token's heads
together), dealt out in random order; what belongs to no sequence holds NaN.
"""
import math

import numpy as np
import torch

from gemv_projection_layers_gb300 import binding as B

DT = {"bf16": (torch.bfloat16, B.PROJ_BF16, 2.0 ** -8), "fp16": (torch.float16, B.PROJ_FP16, 2.0 ** -11)}
FORMATS = {"rows": B.PROJ_KV_ROWS, "e4m3": B.PROJ_KV_E4M3, "int8": B.PROJ_KV_INT8}
TOP = {"e4m3": 448.0, "int8": 127.0}


def quantise(x, fmt):
    """Codes (as their torch type) and scales of rows x, by the format's definition in fp32 on the CPU."""
    x = x.float().cpu()
    amax = x.abs().amax(-1)
    scale = torch.clamp(amax / torch.tensor(TOP[fmt]), min=2.0 ** -126)
    good = torch.isfinite(amax)
    inv = torch.where(good, torch.tensor(1.0) / scale, torch.tensor(0.0))
    y = torch.where(good[..., None], x * inv[..., None], torch.tensor(0.0))
    code = y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().to(torch.int8)
    return code, torch.where(good, scale, torch.tensor(math.nan))


class Cache:
    more = 0  # positions for which every table has room beyond what its sequences need

    def __init__(self, fmt, dtype, lens, kv, D, page, layout="head", seed=0, spare=2):
        self.fmt, self.dtype, self.kv, self.D, self.page = fmt, dtype, kv, D, page
        self.gen = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.width = max(need + [1]) + 1 + -(-self.more // page)
        self.pages = sum(need) + spare
        deal = torch.randperm(self.pages, generator=self.gen).to(torch.int32)
        self.table = torch.full((max(len(lens), 1), self.width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = deal[at:at + n]
            at += n
        torch_type = {"rows": DT[dtype][0], "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[fmt]
        shape = (self.pages, kv, page, D) if layout == "head" else (self.pages, page, kv, D)
        fill = 0 if fmt == "int8" else math.nan
        self.t = {}
        for n in ("k", "v"):
            whole = torch.full(shape, fill, dtype=torch.float32).to(torch_type).cuda()
            self.t[n] = whole if layout == "head" else whole.transpose(1, 2)  # [pages, kv, page, D] either way
            if fmt != "rows":
                self.t[n + "_scale"] = torch.full((self.pages, kv, page), math.nan, device="cuda")
        self.d_table = self.table.cuda()
        s = self.t["k"].stride()
        self.c = B.kv_cache(format=FORMATS[fmt], dtype=DT[dtype][1], pages=self.pages, page=page, heads=kv, D=D, k=self.t["k"], v=self.t["v"],
                            k_scale=self.t.get("k_scale"), v_scale=self.t.get("v_scale"), page_stride=s[0], head_stride=s[1],
                            token_stride=s[2], table=self.d_table, ldt=self.width, width=self.width, sequences=len(lens))

    def spots(self, b, first, n):
        p = torch.arange(first, first + n)
        return self.table[b, p // self.page].long(), p % self.page

    def put(self, b, first, k, v):
        """Rows k, v [n, kv, D] at positions first .. of sequence b, by the plain definition."""
        page, spot = (i.cuda() for i in self.spots(b, first, k.shape[0]))
        for n, x in (("k", k), ("v", v)):
            if self.fmt == "rows":
                self.t[n][page, :, spot] = x.to(self.t[n].dtype).cuda()
            else:
                code, scale = quantise(x, self.fmt)
                raw = self.t[n].view(torch.uint8) if self.fmt == "e4m3" else self.t[n]
                raw[page, :, spot] = (code.view(torch.uint8) if self.fmt == "e4m3" else code).cuda()
                self.t[n + "_scale"][page, :, spot] = scale.cuda()

    def get(self, n, b, first, count):
        """The values [count, kv, D] in 64 bits."""
        page, spot = self.spots(b, first, count)
        x = self.t[n].cpu().float().double()[page, :, spot]
        return x if self.fmt == "rows" else x * self.t[n + "_scale"].cpu().double()[page, :, spot][..., None]

    def raw(self):
        """Everything that the cache holds, as bytes."""
        return {n: t.cpu().contiguous().view(torch.uint8).clone() for n, t in self.t.items()}


def int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets_of(counts):
    return int32(np.concatenate([[0], np.cumsum(counts)]).astype(np.int64).tolist())


def words_of(sees):
    """Rows of truth values [rows, drafts] as 32-bit words."""
    rows, n = sees.shape
    words = max(1, -(-n // 32))
    full = np.zeros((rows, words * 32), np.uint64)
    full[:, :n] = sees
    packed = (full.reshape(rows, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.from_numpy(packed.astype(np.uint32).view(np.int32).copy()).cuda()


def attention(q, k, v, sees, scale):
    """out and lse of one sequence, [rows, heads, D] and [rows, heads], and what the error bounds need: sum of p |v|, and the
    largest sum of |q k| scale.  q [rows, heads, D], k, v [keys, kv, D], sees [rows, keys]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    rows, heads, D = q.shape
    G = heads // k.shape[1]
    out, mag = np.zeros_like(q), np.zeros_like(q)
    lse, spread = np.full((rows, heads), -np.inf), np.zeros((rows, heads))
    for r in range(rows):
        at = np.flatnonzero(sees[r])
        if not len(at):
            continue
        for j in range(heads):
            kk, vv = k[at, j // G], v[at, j // G]
            with np.errstate(invalid="ignore", over="ignore"):
                s = kk @ q[r, j] * scale
                top = s.max()
                p = np.exp(s - top)
                total = p.sum()
                out[r, j] = p @ vv / total
                mag[r, j] = p @ np.abs(vv) / total
                lse[r, j] = top + np.log(total)
                spread[r, j] = (np.abs(kk) @ np.abs(q[r, j])).max() * abs(scale)
    return out, lse, mag, spread
