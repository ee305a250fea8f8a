"""A K/V block pool held in 4 bits, and rotary positions with several axes, as cases that can be timed and compared:
store (new rows quantised into the pool's blocks and read back as the pool holds them), gather (whole contexts read
back dense), attend (softmax attention of the new tokens over the 4-bit blocks), rotate (rows of q and k turned by
their positions) and rotated (q turned in place of a copy, k turned on its way into the pool, v beside it).

Each operator is here twice: in its plain form (elementary torch operations in 32 bits, angles in 64) and, with `own`
set, as the call of liblsc that a user makes.  `exact` states the same results once more in 64 bits.

A 4-bit row of a head is head_dim codes (two a byte, the lower nibble first) and a scale byte for each 16 elements.  A
code is a sign and one of MAGNITUDES; a scale byte b is the 16-bit float of bits b << 7 (5 exponent and 3 mantissa
bits).  A group's scale is the smallest that brings its largest magnitude to 6 or less, and each element takes the
nearest code, ties to the even one.

Batch of a case: sequence i brings n_i new tokens (rows cu[i] .. cu[i+1]) and has kv_i tokens in the cache, the new
ones included, so new token j of it sits at position kv_i - n_i + j; position p is row p % block of block
table[i][p // block].  The lengths depend on the case alone, the values and the placement of blocks on the seed.
"""
import math

import numpy as np
import torch

own = False

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TOP_SCALE = 226  # 10240: six times it is the largest magnitude a 16-bit float takes as a product
SPARE = 7  # blocks of the pool that no sequence uses


def case_(name, op, dtype, kv_heads, head_dim, block, seqs, new, old, q_heads=0, causal=True, singles=0, slack=512, lens=1,
          rotary=0, axes=0, paired=False, mixed_axes=False, far=0):
    """`new`, `old`: (lowest, highest) new tokens and cached tokens of a sequence; the first `singles` sequences
    bring one new token each whatever `new` says.  rotate, rotated: the leading `rotary` elements of a head are turned;
    `axes` position axes, dealt out in turn (`mixed_axes`) or in consecutive sections; neighbours (`paired`) or halves;
    positions up to some thousands behind `far`."""
    c = {"op": op, "dtype": dtype, "kv_heads": kv_heads, "head_dim": head_dim, "block": block, "seqs": seqs,
         "new_lo": new[0], "new_hi": new[1], "old_lo": old[0], "old_hi": old[1], "q_heads": q_heads, "causal": causal,
         "singles": singles, "slack": slack, "lens": lens, "rotary": rotary, "axes": axes, "paired": paired,
         "mixed_axes": mixed_axes, "far": far}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a decode step's new rows of 64 sequences stored, and read back as later steps will see them (launch-bound)
        case_("store_decode", "store", "bf16", 2, 256, 64, 64, (1, 1), (64, 2048)),
        # a resumed prefill of 64 sequences stored and read back
        case_("store_prefill", "store", "bf16", 2, 256, 64, 64, (64, 2048), (0, 2048), slack=256),
        # one sequence's cached prefix read back for inspection or transfer, 16-token blocks, f16
        case_("gather_one", "gather", "f16", 8, 128, 16, 1, (1000, 1000), (0, 0), slack=0),
        # whole contexts of a batch read back
        case_("gather_batch", "gather", "bf16", 8, 128, 64, 24, (900, 16000), (0, 500), slack=0),
        # one user's decode token over a short context (latency)
        case_("decode_one", "attend", "bf16", 2, 256, 64, 1, (1, 1), (1000, 1000), 16),
        # a large decode batch over ragged contexts of 8 heads
        case_("decode_batch", "attend", "bf16", 8, 128, 64, 128, (1, 1), (500, 8000), 32, slack=0),
        # resumed prefill after a restore: ragged continuations over restored prefixes, and decode rows beside them
        case_("chunk_mixed", "attend", "bf16", 2, 256, 64, 24, (64, 2048), (64, 8192), 16, singles=12),
        # one long chunk over a long context, f16
        case_("chunk_long", "attend", "f16", 8, 128, 64, 1, (4096, 4096), (28000, 28000), 32),
        # a decode step's q and k rows, a quarter of each head turned, three axes dealt out in turn
        case_("rotate_decode", "rotate", "bf16", 2, 256, 64, 64, (1, 1), (64, 2048), 16, rotary=64, axes=3, mixed_axes=True,
              far=100000),
        # the prompt of a long video: time, height and width in consecutive sections, whole heads
        case_("rotate_video", "rotate", "bf16", 8, 128, 64, 1, (30011, 30011), (0, 0), 32, rotary=128, axes=3),
        # a decode step's rows turned and appended
        case_("rotated_decode", "rotated", "bf16", 2, 256, 64, 64, (1, 1), (64, 2048), 16, rotary=64, axes=3, mixed_axes=True),
        # a resumed prefill's rows turned and appended
        case_("rotated_prefill", "rotated", "bf16", 2, 256, 64, 64, (64, 2048), (0, 2048), 16, rotary=64, axes=3,
              mixed_axes=True, slack=0),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "gather", "attend", "attend", "attend", "attend", "rotate", "rotated"])
    dtype = rng.choice(["bf16", "bf16", "f16"] + (["f32"] if op in ("store", "rotate") else []))
    head_dim = rng.choice([64, 128, 256] + ([80, 96] if op != "attend" else []))
    kv_heads = rng.choice([1, 2, 3, 4, 8] if head_dim < 256 else [1, 2, 4])
    group = 0 if op in ("store", "gather") else rng.choice([1, 2, 4, 5, 7, 8])
    block = rng.choice([16, 32, 64, 64, 128, 48, 24])
    seed, slack = rng.randrange(1 << 20), rng.choice([0, 16, 256, 512])
    rotary = axes = far = 0
    paired = mixed = False
    if op in ("rotate", "rotated"):
        rotary = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4])
        axes, far = rng.choice([1, 2, 3, 3, 4]), rng.choice([0, 0, 1000, 1000000])
        paired, mixed = rng.random() < 0.4, rng.random() < 0.5
    kind = rng.choice(["decode", "chunk", "mixed"])
    if kind == "decode":
        seqs, new, top = log_int(rng, 1, 160), (1, rng.choice([1, 1, 1, 2, 4])), log_int(rng, 100, 12000)
    else:
        seqs, top = log_int(rng, 1, 16), log_int(rng, 100, 12000)
        new = (log_int(rng, 1, 64), log_int(rng, 64, 1500))
    old = (rng.randrange(0, max(1, top // 2)), top)
    singles, causal = (seqs // 2 if kind == "mixed" else 0), rng.random() < 0.8
    while True:  # fewer sequences until it costs no more than the largest listed cases
        c = case_("", op, dtype, kv_heads, head_dim, block, seqs, new, old, kv_heads * group, causal=causal,
                  singles=min(singles, seqs // 2), slack=slack, lens=seed, rotary=rotary, axes=axes, paired=paired,
                  mixed_axes=mixed, far=far)
        w = work(c)
        if seqs == 1 or (w["bytes"] < 0.5e9 and w["flops"] < 1.0e12):
            return c
        seqs = max(1, seqs * 3 // 4)


def lengths(c):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    r = np.random.RandomState(c["lens"])
    n = r.randint(c["new_lo"], c["new_hi"] + 1, c["seqs"])
    n[:c["singles"]] = 1
    old = r.randint(c["old_lo"], c["old_hi"] + 1, c["seqs"])
    return n.astype(np.int64), (n + old).astype(np.int64)


def in_four_bits(c):
    return c["op"] in ("store", "gather", "attend")


def layout(c):
    """The offset of a block's scales (4 bits: one byte per 16 elements) and the page stride."""
    rows = c["block"] * c["kv_heads"]
    codes = rows * c["head_dim"] // 2 if in_four_bits(c) else rows * c["head_dim"] * BYTES[c["dtype"]]
    scales = (codes + 15) // 16 * 16
    payload = scales + rows * c["head_dim"] // 16 if in_four_bits(c) else codes
    return scales, (payload + 15) // 16 * 16 + c["slack"]


def axis_of_pair(c):
    """The axis that each of the rotary / 2 pairs takes its position from."""
    i = np.arange(c["rotary"] // 2)
    return (i % c["axes"] if c["mixed_axes"] else i * c["axes"] // (c["rotary"] // 2)).astype(np.uint8)


def frequencies(c):
    return 10000.0 ** (-np.arange(0, c["rotary"], 2, dtype=np.float64) / c["rotary"])


def inputs(c, seed):
    """The pool's buffer ([K lane][V lane], num_blocks pages each), the batch and the dense inputs, on the GPU."""
    n, kv = lengths(c)
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, D, T, dt = c["kv_heads"], c["head_dim"], int(n.sum()), TORCH[c["dtype"]]
    gain = torch.exp(0.5 * torch.randn(H, D, generator=g, device="cuda"))  # K's channels differ in size
    s = {"case": c, "T": T}
    if c["axes"]:
        # runs of text (every axis the same) between frames of 20 x 30: one time, rows and columns
        t = torch.arange(T, device="cuda")
        shot, at = t // 700, t % 700
        time = torch.where(at < 100, at, 100 + shot)
        up, across = torch.where(at < 100, at, 100 + (at - 100) // 30), torch.where(at < 100, at, 100 + (at - 100) % 30)
        start = c["far"] + 37 * shot + int(torch.randint(0, 100, (1,), generator=g, device="cuda"))
        s["positions"] = torch.stack([start + [time, up, across][a % 3] for a in range(c["axes"])]).to(torch.int32)
    if c["op"] == "rotate":
        s["x"] = torch.randn(T, c["q_heads"] + H, D, generator=g, device="cuda").to(dt)
        return s
    per = -(-kv // c["block"])
    blocks = int(per.sum()) + SPARE
    scales, page = layout(c)
    s.update(blocks=blocks, page=page, scale_off=scales)
    s["buf"] = torch.zeros(2 * blocks * page, dtype=torch.uint8, device="cuda")
    if c["op"] in ("gather", "attend"):
        # every block holds rows, the ones behind a sequence's last too: those are left from earlier use
        for lane, by in enumerate((gain, None)):
            step = max(1, 2 ** 25 // (c["block"] * H * D))
            for b in range(0, blocks, step):
                x = torch.randn(min(step, blocks - b), c["block"], H, D, generator=g, device="cuda")
                codes, scale = quantise(x if by is None else x * by)
                codes_of(s, lane)[b:b + len(x)] = codes
                scales_of(s, lane)[b:b + len(x)] = scale
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    at = np.concatenate([[0], np.cumsum(per)])
    table = np.zeros((c["seqs"], int(per.max())), np.int64)
    used = np.arange(table.shape[1])[None] < per[:, None]
    table[used] = (at[:-1, None] + np.arange(table.shape[1])[None])[used]
    s["table"] = torch.where(torch.from_numpy(used).cuda(), order[torch.from_numpy(table).cuda()], 0).to(torch.int32)
    s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    s["kv"] = torch.from_numpy(kv.astype(np.int32)).cuda()
    if c["op"] in ("store", "rotated"):
        s["k"] = (torch.randn(T, H, D, generator=g, device="cuda") * gain).to(dt)
        s["v"] = torch.randn(T, H, D, generator=g, device="cuda").to(dt)
    if c["op"] in ("attend", "rotated"):
        s["q"] = (2 * torch.randn(T, c["q_heads"], D, generator=g, device="cuda")).to(dt)
        s["scale"] = 1.0 / math.sqrt(D)
    return s


def codes_of(s, lane):
    """Codes of a lane as bytes [blocks, block, kv_heads, head_dim / 2], through the page stride."""
    c = s["case"]
    B, H, W = c["block"], c["kv_heads"], c["head_dim"] // 2
    return s["buf"].as_strided((s["blocks"], B, H, W), (s["page"], H * W, W, 1), lane * s["blocks"] * s["page"])


def scales_of(s, lane):
    c = s["case"]
    B, H, W = c["block"], c["kv_heads"], c["head_dim"] // 16
    return s["buf"].as_strided((s["blocks"], B, H, W), (s["page"], H * W, W, 1),
                               lane * s["blocks"] * s["page"] + s["scale_off"])


def rows_of(s, lane):
    """Rows of a lane of a pool of the dense type, [blocks, block, kv_heads, head_dim]."""
    c = s["case"]
    t = s["buf"].view(TORCH[c["dtype"]])
    stride = s["page"] // BYTES[c["dtype"]]
    return t.as_strided((s["blocks"], c["block"], c["kv_heads"], c["head_dim"]),
                        (stride, c["kv_heads"] * c["head_dim"], c["head_dim"], 1), lane * s["blocks"] * stride)


def scale_value(byte):
    """A scale byte's value in 32 bits: the 16-bit float of bits byte << 7."""
    return (byte.to(torch.int16) << 7).view(torch.float16).float()


def quantise(x):
    """[..., head_dim] -> bytes of codes [..., head_dim / 2] and scale bytes [..., head_dim / 16].  Six times a scale and
    a tie times a scale have seven bits at most, so every comparison is exact in 32 bits."""
    x = x.float().unflatten(-1, (-1, 16))
    top = x.abs().amax(-1)
    ladder = 6 * scale_value(torch.arange(TOP_SCALE + 1, device=x.device))
    byte = torch.searchsorted(ladder, top.contiguous()).clamp(max=TOP_SCALE)  # the first scale with 6 s >= top
    s, a = scale_value(byte)[..., None], x.abs()
    code = torch.zeros_like(x, dtype=torch.uint8)
    for tie, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= tie * s) if up else (a > tie * s)
    code = torch.where(byte[..., None] > 0, code + 8 * torch.signbit(x), 0).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, byte.to(torch.uint8)


def prepare(case, seed):
    s = inputs(case, seed)
    if own:
        from linear_attention_state_lsc_gb300 import lsc as L

        c, T = case, s["T"]
        code, s["L"] = {"bf16": L.LSC_BF16, "f16": L.LSC_F16, "f32": L.LSC_F32}[c["dtype"]], L
        if c["axes"]:
            turn = L.rotary(c["rotary"], s["positions"], frequencies(c), pair_axis=axis_of_pair(c), interleaved=c["paired"])
        if c["op"] == "rotate":
            s["out"] = torch.empty_like(s["x"])
            s["args"] = L.rotate_args(T, c["q_heads"] + c["kv_heads"], c["head_dim"], code, s["x"], s["out"], turn)
            return s
        kind = L.LSC_E2M1 if in_four_bits(c) else code
        desc = L.lsc_kv_pool_desc(1, s["blocks"], c["block"], c["kv_heads"], c["head_dim"], kind, s["page"])
        rc, pool = L.lsc_kv_pool_create(desc, s["buf"], s["buf"].numel())
        assert rc == L.LSC_OK, L.lsc_error_string(rc)
        s["pool"] = Pool(L, pool)
        n, kv = lengths(c)
        batch = L.kv_batch(c["seqs"], T, s["table"], s["cu"], s["kv"], max_blocks=s["table"].shape[1])
        dt = TORCH[c["dtype"]]
        if c["op"] in ("store", "gather"):
            s["k_out"], s["v_out"] = (torch.empty(T, c["kv_heads"], c["head_dim"], dtype=dt, device="cuda") for _ in "kv")
            s["back"] = L.kv_gather_args(batch, s["k_out"], s["v_out"], code)
        if c["op"] == "store":
            s["args"] = L.kv_append_args(batch, s["k"], s["v"], code)
        elif c["op"] == "rotated":
            s["q_out"] = torch.empty_like(s["q"])
            s["args"] = L.kv_append_rotated_args(L.kv_append_args(batch, s["k"], s["v"], code), turn, c["q_heads"], s["q"],
                                                 s["q_out"])
        elif c["op"] == "attend":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(T, c["q_heads"], device="cuda")
            bounds = dict(causal=c["causal"], max_seq_tokens=int(n.max()), max_kv_tokens=int(kv.max()))
            a = L.kv_attend_args(batch, c["q_heads"], s["q"], s["out"], code, s["scale"], lse=s["lse"], **bounds)
            rc, need = L.lsc_kv_attend_workspace_bytes(pool, a)
            assert rc == L.LSC_OK, L.lsc_error_string(rc)
            s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
            s["args"] = L.kv_attend_args(batch, c["q_heads"], s["q"], s["out"], code, s["scale"], lse=s["lse"],
                                         workspace=s["workspace"], workspace_bytes=need, **bounds)
    return s


class Pool:
    """A pool handle that lives as long as the state that holds it."""

    def __init__(self, lib, handle):
        self.lib, self.handle = lib, handle

    def __del__(self):
        self.lib.lsc_kv_pool_destroy(self.handle)


def run(s):
    c = s["case"]
    if own:
        own_run(s)
    else:
        PLAIN[c["op"]](s)
    if c["op"] in ("store", "gather"):
        return [s["k_out"], s["v_out"]]
    if c["op"] == "attend":
        return [s["out"], s["lse"]]
    return s["out"] if c["op"] == "rotate" else [s["q_out"], rows_of(s, 0), rows_of(s, 1)]


def own_run(s):
    op, L, stream = s["case"]["op"], s["L"], torch.cuda.current_stream()
    if op == "rotate":
        rc = L.lsc_rotate(s["args"], stream)
    elif op == "rotated":
        rc = L.lsc_kv_append_rotated(s["pool"].handle, 0, s["args"], stream)
    elif op == "attend":
        rc = L.lsc_kv_attend(s["pool"].handle, 0, s["args"], stream)
    else:
        rc = L.lsc_kv_append(s["pool"].handle, 0, s["args"], stream) if op == "store" else L.LSC_OK
        if rc == L.LSC_OK:
            rc = L.lsc_kv_gather(s["pool"].handle, 0, s["back"], stream)
    if rc != L.LSC_OK:
        raise L.LscError(rc, op)


def places(s):
    """Of each new token: its sequence, block and row."""
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=s["T"])
    pos = s["kv"].long()[seq] - n[seq] + torch.arange(s["T"], device="cuda") - s["cu"].long()[seq]
    block = s["case"]["block"]
    return seq, s["table"].long()[seq, pos // block], pos % block


def values(s, lane, *at):
    """Rows of a lane of a 4-bit pool in 32 bits."""
    b = codes_of(s, lane)[at]
    code = torch.stack([b & 15, b >> 4], -1).flatten(-2).long()
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device="cuda")
    return (table[code].unflatten(-1, (-1, 16)) * scale_value(scales_of(s, lane)[at])[..., None]).flatten(-2)


def plain_store(s):
    _, block, row = places(s)
    for lane, x in enumerate((s["k"], s["v"])):
        codes_of(s, lane)[block, row], scales_of(s, lane)[block, row] = quantise(x)
    plain_gather(s)


def plain_gather(s):
    _, block, row = places(s)
    dt = TORCH[s["case"]["dtype"]]
    s["k_out"], s["v_out"] = values(s, 0, block, row).to(dt), values(s, 1, block, row).to(dt)


def plain_attend(s):
    """Every sequence padded to the longest: scores, masked, exponentials over their sum, weighted values."""
    c = s["case"]
    H, D, S = c["kv_heads"], c["head_dim"], c["seqs"]
    G = c["q_heads"] // H
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    N = c["new_hi"] if c["singles"] < S else 1
    seq, _, _ = places(s)
    j = torch.arange(s["T"], device="cuda") - s["cu"].long()[seq]
    q = torch.zeros(S, N, H, G, D, device="cuda")
    q[seq, j] = s["q"].float().view(-1, H, G, D) * s["scale"]
    table = s["table"].long()
    k = values(s, 0, table).view(S, -1, H, D)
    p = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(S, H, G * N, D), k.permute(0, 2, 3, 1)).view(S, H, G, N, -1)
    del k, q
    key = torch.arange(p.shape[-1], device="cuda")
    last = s["kv"].long()[:, None].expand(S, N) - 1
    if c["causal"]:
        last = (last + 1 - n[:, None] + torch.arange(N, device="cuda")).clamp(max=last)
    p.masked_fill_((key > last[..., None])[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(top.clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    v = values(s, 1, table).view(S, -1, H, D).permute(0, 2, 1, 3)
    o = torch.matmul(p.view(S, H, G * N, -1), v).view(S, H, G, N, D) / total.clamp(min=1e-30)
    lse = (top + total.log())[..., 0]
    s["out"] = o.permute(0, 3, 1, 2, 4)[seq, j].reshape(s["T"], c["q_heads"], D).to(TORCH[c["dtype"]])
    s["lse"] = lse.permute(0, 3, 1, 2)[seq, j].reshape(s["T"], c["q_heads"])


def turned(s, x):
    """[T, heads, head_dim] in the dense type -> turned, in 32 bits; the angles in 64."""
    c = s["case"]
    half = c["rotary"] // 2
    axis = torch.from_numpy(axis_of_pair(c).astype(np.int64)).cuda()
    angle = s["positions"].double()[axis].T * torch.from_numpy(frequencies(c)).cuda()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    out = x.clone()
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["paired"] else (slice(0, half), slice(half, 2 * half))
    out[..., one] = x[..., one] * cos - x[..., two] * sin
    out[..., two] = x[..., two] * cos + x[..., one] * sin
    return out


def plain_rotate(s):
    s["out"] = turned(s, s["x"]).to(TORCH[s["case"]["dtype"]])


def plain_rotated(s):
    _, block, row = places(s)
    dt = TORCH[s["case"]["dtype"]]
    s["q_out"] = turned(s, s["q"]).to(dt)
    rows_of(s, 0)[block, row] = turned(s, s["k"]).to(dt)
    rows_of(s, 1)[block, row] = s["v"]


PLAIN = {"store": plain_store, "gather": plain_gather, "attend": plain_attend, "rotate": plain_rotate,
         "rotated": plain_rotated}


def work(case):
    c = case
    n, kv = lengths(c)
    H, D, T, es = c["kv_heads"], c["head_dim"], int(n.sum()), BYTES[c["dtype"]]
    held = D // 2 + D // 16  # bytes of a 4-bit row
    where = 4.0 * c["axes"] * T
    if c["op"] == "store":
        return {"bytes": 2.0 * H * T * (2 * D * es + held), "flops": 0.0}
    if c["op"] == "gather":
        return {"bytes": 2.0 * H * T * (held + D * es), "flops": 0.0}
    if c["op"] == "rotate":
        return {"bytes": 2.0 * T * (c["q_heads"] + H) * D * es + where, "flops": 3.0 * T * (c["q_heads"] + H) * c["rotary"]}
    if c["op"] == "rotated":
        return {"bytes": 2.0 * T * (c["q_heads"] + 2 * H) * D * es + where,
                "flops": 3.0 * T * (c["q_heads"] + H) * c["rotary"]}
    seen = n * (kv - n) + n * (n + 1) // 2 if c["causal"] else n * kv
    dense = T * c["q_heads"] * (2 * D * es + 4)
    return {"bytes": 2.0 * H * held * int(kv.sum()) + dense, "flops": 4.0 * D * c["q_heads"] * int(seen.sum())}


def exact(case, seed):
    """Each result from its definition, a sequence and a head at a time, in 64 bits."""
    c, s = case, inputs(case, seed)
    n, kv = lengths(c)
    H, D, B = c["kv_heads"], c["head_dim"], c["block"]
    cu = np.concatenate([[0], np.cumsum(n)])
    if c["axes"]:
        # a pair as a complex number, turned by a product with exp(i angle)
        where = s["positions"].double()[torch.from_numpy(axis_of_pair(c).astype(np.int64)).cuda()].T
        spin = torch.polar(torch.ones_like(where), where * torch.from_numpy(frequencies(c)).cuda())

        def spun(x):
            x, r = x.double(), c["rotary"]
            if c["paired"]:
                z = torch.view_as_complex(x[..., :r].unflatten(-1, (-1, 2)).contiguous()) * spin[:, None]
                head = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * spin[:, None]
                head = torch.cat([z.real, z.imag], -1)
            return torch.cat([head, x[..., r:]], -1)

        if c["op"] == "rotate":
            return spun(s["x"])
    pages, blocks = s["buf"].view(2, s["blocks"], s["page"]), s["blocks"]
    table = s["table"].cpu().numpy()

    def at(seq, lo, hi):
        p = np.arange(lo, hi)
        return torch.from_numpy(table[seq][p // B].astype(np.int64)).cuda(), torch.from_numpy(p % B).cuda()

    if c["op"] == "rotated":
        lanes = []
        for x in (spun(s["k"]), s["v"].double()):
            put = torch.zeros(blocks, B, H, D, dtype=torch.float64, device="cuda")
            for i in range(c["seqs"]):
                put[at(i, int(kv[i] - n[i]), int(kv[i]))] = x[cu[i]:cu[i + 1]]
            lanes.append(put)
        return [spun(s["q"]), *lanes]

    def grid(x):
        """Values [..., D] as a 4-bit row holds them, from the value's own power of two."""
        x = x.double().unflatten(-1, (-1, 16))
        want = x.abs().amax(-1, keepdim=True) / 6
        # scales have steps of an eighth of their power of two, of 2^-17 below 2^-14
        step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -14))) - 3)
        scale = (torch.ceil(want / step) * step).clamp(max=10240.0)
        y = x / torch.where(scale > 0, scale, 1.0)
        # codes have steps of half their power of two, of 1/2 below 1; ties go to the even one
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1.0))) - 1)
        return ((torch.round(y / step) * step).clamp(-6, 6) * scale).flatten(-2)

    if c["op"] == "store":
        return [grid(s["k"]), grid(s["v"])]

    def held(lane, seq, lo, hi):
        """Positions [lo, hi) of a sequence: values [hi - lo, H, D]."""
        b, r = at(seq, lo, hi)
        raw = pages[lane][:, :B * H * D // 2].view(blocks, B, H, D // 2)[b, r].long()
        up = pages[lane][:, s["scale_off"]:s["scale_off"] + B * H * D // 16].view(blocks, B, H, D // 16)[b, r].long()
        x = torch.stack([raw % 16, raw // 16], -1).flatten(-2)
        e, m = x % 8 // 2, x % 2
        x = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double())) * (1 - 2 * (x // 8))
        e, m = up // 8, up % 8
        up = torch.where(e == 0, m * 2.0 ** -17, (8 + m) * torch.exp2((e - 18).double()))
        return (x.unflatten(-1, (-1, 16)) * up[..., None]).flatten(-2)

    if c["op"] == "gather":
        return [torch.cat([held(lane, i, int(kv[i] - n[i]), int(kv[i])) for i in range(c["seqs"])]) for lane in (0, 1)]
    G = c["q_heads"] // H
    if work(c)["flops"] > 5e12:
        return None
    out = torch.zeros(s["T"], c["q_heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], c["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for i in range(c["seqs"]):
        k, v = held(0, i, 0, int(kv[i])), held(1, i, 0, int(kv[i]))
        q = s["q"][cu[i]:cu[i + 1]].double()
        ahead = torch.arange(int(kv[i]), device="cuda")[None] > torch.arange(int(n[i]), device="cuda")[:, None] + int(kv[i] - n[i])
        for h in range(c["q_heads"]):
            z = q[:, h] @ k[:, h // G].T / math.sqrt(D)
            if c["causal"]:
                z[ahead] = -math.inf
            l = torch.logsumexp(z, 1)
            lse[cu[i]:cu[i + 1], h] = l
            out[cu[i]:cu[i + 1], h] = torch.exp(z - l[:, None]) @ v[:, h // G]
    return [out, lse]
