"""GPU tests of the vocabulary operators (4-bit logits, log probabilities and
their gradient, embedding and its gradient) against the float64 oracle.

Every tolerance is an error bound of the FP32 computation, in units of
u = 2^-24 (half a step of FP32), plus half a step of the output type."""
import numpy as np
import pytest

import lm_head_gumbel_amd as fs
from oracle import vocab as OV
from gpu_util import dev, host, log, torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}    # steps below the normal range


def tdt(name):
    t = torch()
    return {"f32": t.float32, "bf16": t.bfloat16, "f16": t.float16}[name]


def as_type(a, name):
    """Device tensor of element type `name`, and its exact float64 values."""
    x = dev(np.asarray(a, np.float32)).to(tdt(name))
    return x, host(x.float()).astype(np.float64)


def f64(x):
    return host(x.float()).astype(np.float64)


def garbage(nbytes):
    t = torch()
    return t.full((max(1, nbytes),), 0xC3, dtype=t.uint8, device="cuda")


# ---------------------------------------------------------------------------
# 4-bit logits
# ---------------------------------------------------------------------------
def quant_problem(B, d, V, group, sdt, zero, seed=0, zlo=0, zhi=16):
    rng = np.random.default_rng(seed)
    H, Hf = as_type(rng.normal(size=(B, d)), "bf16")
    q = rng.integers(0, 256, (V, d // 2), dtype=np.uint8)
    S, Sf = as_type(0.01 * np.exp(0.5 * rng.normal(size=(V, d // group))) * rng.choice([-1, 1], (V, d // group)), sdt)
    z = rng.integers(zlo, zhi, (V, d // group), dtype=np.uint8) if zero else None
    return H, Hf, q, S, Sf, z


def quant_bound(Hf, q, Sf, z, group):
    """|error| of a logit: each group's sum runs over at most 128 products of
    h with a weight offset by up to 32 (the offset is taken back with the
    group's sum of h), the groups' scaled sums are added one by one; a matrix
    instruction may truncate instead of rounding (two u a step)."""
    d = Hf.shape[1]
    n = OV.unpack_w4(q).astype(np.float64) + 32 + (8.0 if z is None else np.repeat(z.astype(np.float64), group, 1))
    mag = np.abs(Hf) @ (n * np.repeat(np.abs(Sf), group, 1)).T
    return 2 * U * (min(group, 128) + d / min(group, 128) + 16) * mag


@pytest.mark.parametrize("B,d,V,group,sdt,zero", [
    (1, 32, 1, 32, "f32", False), (3, 64, 17, 32, "bf16", True), (4, 256, 4096, 32, "f32", False),
    (16, 96, 100, 32, "f16", True), (17, 192, 333, 64, "bf16", False), (2, 64, 5, 64, "f32", True),
    (32, 128, 50, 128, "f16", True), (5, 640, 1000, 128, "bf16", True), (33, 256, 129, 256, "f32", False),
    (64, 384, 77, 128, "f16", False), (65, 128, 200, 64, "bf16", True), (130, 512, 96, 512, "f32", True),
    (1, 4096, 2000, 128, "bf16", True), (20, 5120, 300, 128, "f16", False), (48, 2048, 515, 64, "bf16", True),
    (7, 4096, 515, 32, "f32", True), (64, 2080, 300, 32, "bf16", False), (300, 160, 60, 32, "f16", True),
    (16, 8192, 600, 128, "bf16", True), (24, 8192, 200, 32, "f32", True), (18, 6144, 200, 64, "f16", True),
    (5, 1024, 300, 64, "bf16", True), (12, 1152, 100, 32, "f16", True), (2, 2048, 9000, 64, "f32", False),
    (30, 1024, 9000, 32, "bf16", True), (64, 1024, 9000, 128, "f32", True), (50, 640, 20000, 64, "bf16", True)])
def test_quant_logits_match_the_oracle(B, d, V, group, sdt, zero):
    H, Hf, q, S, Sf, z = quant_problem(B, d, V, group, sdt, zero, seed=B + d)
    t = torch()
    out = t.full((B + 1, V), 7.0, device="cuda")
    W = fs.quant(dev(q), S, None if z is None else dev(z), group)
    log(f"quant B={B} d={d} V={V} group={group} {sdt} zero={zero}")
    fs.check(fs.fs_logits_quant(fs.params(B, d, V), H, W, out[:B]), "fs_logits_quant")
    t.cuda.synchronize()
    want = Hf @ OV.dequantise(q, Sf, z, group).T
    err = np.abs(f64(out[:B]) - want)
    assert np.all(err <= quant_bound(Hf, q, Sf, z, group))
    assert bool((out[B] == 7.0).all())          # the row behind the last is left as it was


def test_quant_zero_points_use_the_whole_byte():
    H, Hf, q, S, Sf, z = quant_problem(9, 256, 130, 64, "f32", True, seed=5, zlo=0, zhi=256)
    out = torch().empty((9, 130), device="cuda")
    fs.check(fs.fs_logits_quant(fs.params(9, 256, 130), H, fs.quant(dev(q), S, dev(z), 64), out))
    want = Hf @ OV.dequantise(q, Sf, z, 64).T
    assert np.all(np.abs(f64(out) - want) <= quant_bound(Hf, q, Sf, z, 64))


def test_quant_rows_do_not_meet():
    """A row of infinities or NaN in H, or of NaN in the scales, stays in its
    own row or column, and bad shapes past V or B add nothing."""
    B, d, V, group = 5, 256, 33, 128
    H, Hf, q, S, Sf, z = quant_problem(B, d, V, group, "f32", True, seed=6)
    H[3, 7] = float("nan")
    H[1, 200] = float("inf")
    S[32, 1] = float("nan")
    out = torch().empty((B, V), device="cuda")
    fs.check(fs.fs_logits_quant(fs.params(B, d, V), H, fs.quant(dev(q), S, dev(z), group), out))
    got = f64(out)
    rows = [0, 2, 4]
    want = Hf[rows] @ OV.dequantise(q[:32], Sf[:32], z[:32], group).T
    bound = quant_bound(Hf[rows], q[:32], Sf[:32], z[:32], group)
    assert np.all(np.abs(got[rows][:, :32] - want) <= bound)
    assert np.all(np.isnan(got[:, 32])) and np.all(np.isnan(got[3]))
    assert not np.any(np.isfinite(got[1, :32]))


def test_quant_offsets_past_32_bits():
    """W of 2.2e9 bytes: the last rows are read from behind 2^31."""
    t = torch()
    d, group, V, tail = 4096, 128, 1_100_003, 40
    rng = np.random.default_rng(11)
    H, Hf, q, S, Sf, z = quant_problem(2, d, tail, group, "bf16", True, seed=11)
    Q = t.zeros((V, d // 2), dtype=t.uint8, device="cuda")
    SS = t.zeros((V, d // group), dtype=t.bfloat16, device="cuda")
    Z = t.zeros((V, d // group), dtype=t.uint8, device="cuda")
    Q[-tail:], SS[-tail:], Z[-tail:] = dev(q), S, dev(z)
    out = t.full((2, V), 7.0, device="cuda")
    fs.check(fs.fs_logits_quant(fs.params(2, d, V), H, fs.quant(Q, SS, Z, group), out))
    t.cuda.synchronize()
    want = Hf @ OV.dequantise(q, Sf, z, group).T
    assert np.all(np.abs(f64(out[:, -tail:]) - want) <= quant_bound(Hf, q, Sf, z, group))
    assert bool((out[:, :-tail] == 0).all())


# ---------------------------------------------------------------------------
# log probabilities
# ---------------------------------------------------------------------------
class Lp:
    """One problem: device operands and the oracle's view of them."""

    def __init__(self, B, V, dtype="f32", n_top=0, pad=0, temp=None, allow=None, n_valid=None, v_offset=0, seed=0,
                 logits=None, token=None, std=3.0, flags=0):
        t = torch()
        rng = np.random.default_rng(seed)
        self.B, self.V, self.dtype, self.n_top, self.v_offset = B, V, dtype, n_top, v_offset
        a = std * rng.normal(size=(B, V)) if logits is None else logits
        buf = t.full((B, V + pad), float("nan"), dtype=tdt(dtype), device="cuda")
        buf[:, :V] = dev(np.asarray(a, np.float32)).to(tdt(dtype))
        self.logits = buf[:, :V]
        self.values = f64(self.logits)
        tok = rng.integers(0, max(V, 1), B) + v_offset if token is None else np.asarray(token)
        self.token_h = tok
        self.token = dev(tok.astype(np.int32))
        self.temp = None if temp is None else dev(np.asarray(temp, np.float32))
        self.allow_h = allow
        self.allow = None if allow is None else dev(np.asarray(allow, np.uint32).view(np.int32))
        self.p = fs.params(B, 0, V, n_valid=n_valid, v_offset=v_offset, flags=flags)
        self.l = OV.clean_logits(self.values, None if n_valid is None else n_valid - v_offset, allow)
        self.T = OV.row_temps(None if temp is None else np.asarray(temp, np.float32), B, bool(flags))
        self.want = OV.logprobs(self.l, self.T, self.token_h, n_top, v_offset)

    def out(self):
        t = torch()
        f = dict(dtype=t.float32, device="cuda")
        i = dict(dtype=t.int32, device="cuda")
        return dict(logprob=t.full((self.B,), 7.0, **f), rank=t.full((self.B,), -7, **i), lse=t.full((self.B,), 7.0, **f),
                    entropy=t.full((self.B,), 7.0, **f), top_idx=t.full((self.B, self.n_top), -7, **i),
                    top_logprob=t.full((self.B, self.n_top), 7.0, **f))

    def ws(self):
        n = fs.fs_workspace_bytes(self.p, fs.FS_VARIANT_LOGPROBS, self.n_top)
        assert n > 0
        return garbage(n)

    def call(self, o, ws, stream=None):
        fs.check(fs.fs_logprobs(self.p, self.logits, self.temp, self.allow, self.token, self.n_top, o["logprob"], o["rank"],
                                o["lse"], o["entropy"], o["top_idx"], o["top_logprob"], ws, stream=stream), "fs_logprobs")

    def run(self):
        o = self.out()
        self.call(o, self.ws())
        torch().cuda.synchronize()
        return o

    def check(self, o):
        w = self.want
        assert np.array_equal(host(o["rank"]), w["rank"])
        assert np.array_equal(host(o["top_idx"]), w["top_idx"])
        # ln S: 300 additions in a row at most (elements of a thread, threads, slices), each exponential within
        # (2 |x| + 4) u; ln itself 4 u; (l - m) / T 2 u; the last addition u of the result
        s = 304 + 4 * w["absx"]
        small = lambda v: 4 * np.where(np.isfinite(v), np.abs(v), 0)  # noqa: E731
        near(o["lse"], w["lse"], U * (s + small(w["m"]) + small(w["lse"])))
        near(o["logprob"], w["logprob"], U * (s + small(w["logprob"]) + 4 * np.abs(w["lse"] - w["m"], where=np.isfinite(w["lse"]), out=np.zeros(self.B))))
        near(o["top_logprob"], w["top_logprob"], U * (s[:, None] + 2 * small(w["top_logprob"]) + 64))
        # A / S: both sums as above, the terms of A within (2 x^2 + 4 |x|) u
        near(o["entropy"], w["entropy"], U * (s * (1 + 2 * w["absx"]) + 4 * w["x2"] + 64))


def near(got, want, tol):
    got = f64(got)
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin])
    assert np.all(np.abs(got[fin] - want[fin]) <= np.broadcast_to(tol, want.shape)[fin]), \
        (np.abs(got[fin] - want[fin]) - np.broadcast_to(tol, want.shape)[fin]).max()


def some_mask(B, V, seed, keep=2):
    rng = np.random.default_rng(seed)
    a = rng.integers(0, 2 ** 32, (B, (V + 31) // 32), dtype=np.uint64).astype(np.uint32)
    for _ in range(keep - 1):
        a |= rng.integers(0, 2 ** 32, a.shape, dtype=np.uint64).astype(np.uint32)
    return a


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,V,n_top,pad", [(1, 1, 1, 0), (3, 5, 8, 0), (2, 64, 64, 3), (5, 255, 3, 1), (4, 2049, 20, 7),
                                           (7, 8192, 5, 0), (2, 8193, 64, 0), (3, 50257, 20, 0), (70, 1000, 0, 24),
                                           (300, 333, 2, 5), (2, 151936, 20, 0), (40, 33000, 7, 8)])
def test_logprobs_match_the_oracle(B, V, n_top, pad, dtype):
    rng = np.random.default_rng(B + V)
    log(f"logprobs B={B} V={V} n_top={n_top} pad={pad} {dtype}")
    x = Lp(B, V, dtype, n_top, pad, temp=rng.uniform(0.3, 1.7, B) if B % 2 else None, seed=V)
    x.check(x.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logprobs_masks_shards_and_greedy_rows(dtype):
    B, V = 9, 9001
    temp = np.array([1, 0, -1, np.nan, np.inf, 0.05, 30, 1e-30, 0.7])
    allow = some_mask(B, V, 2)
    allow[8] = 0                                   # nothing left
    allow[6] = 0
    allow[6, 100] = 1 << 7                         # one id left: 3207
    token = np.full(B, 160 + 3207)
    token[0], token[1], token[2], token[3] = -1, 159, 160 + V, 160 + V - 1
    for kw in (dict(), dict(n_valid=160 + 8990), dict(n_valid=100), dict(flags=fs.FS_NO_NOISE)):
        log(f"masks {dtype} {kw}")
        x = Lp(B, V, dtype, 12, 5, temp, allow, v_offset=160, token=token, seed=3, **kw)
        o = x.run()
        # T = 1e-30: every id but the best has -inf, T = inf: all equal
        x.check(o)


def test_logprobs_odd_values():
    """+-inf, NaN, the type's extremes, equal values, -0 and 0, a row all -inf."""
    inf, nan, big = np.inf, np.nan, 3.4028235e38
    rows = np.zeros((10, 40), np.float32)
    rows[0] = -inf
    rows[1] = nan
    rows[2] = -big                                  # the lowest value as a mask, everywhere
    rows[3, :20] = -big                             # and on half of the row
    rows[4, 5] = inf
    rows[5, 5] = rows[5, 9] = inf
    rows[6, ::2] = -0.0                             # equal: the lower id first
    rows[7, 3] = -inf
    rows[7, 4] = nan
    rows[8] = np.linspace(-50, 50, 40)
    rows[9] = 1e30
    for tok in (0, 5, 9, 39):
        x = Lp(10, 40, "f32", 7, logits=rows, token=np.full(10, tok))
        o = x.run()
        x.check(o)
    assert host(o["top_idx"])[6].tolist() == list(range(7))
    assert host(o["lse"])[0] == -inf and host(o["lse"])[1] == -inf
    assert host(o["entropy"])[:2].tolist() == [0, 0]


@pytest.mark.parametrize("V", [7000, 151936])
def test_logprobs_alternatives_of_adverse_rows(V):
    """Ascending, descending, all equal, few values, and all the best in one
    place: the selection has to hold for every order."""
    rng = np.random.default_rng(0)
    rows = np.zeros((7, V), np.float32)
    rows[0] = np.arange(V) * 1e-3
    rows[1] = -np.arange(V) * 1e-3
    rows[3] = rng.integers(0, 3, V)
    rows[4] = rng.normal(size=V)
    rows[4, 4000:4100] += 20
    rows[5] = -np.inf
    rows[5, V // 2:V // 2 + 9] = 1.0
    rows[6, V - 70:] = 5
    for n in (1, 20, 64):
        x = Lp(7, V, "f32", n, logits=rows, token=np.array([V - 1, V - 1, V - 1, V // 2, 4050, V // 2 + 4, V - 1]))
        x.check(x.run())


def test_logprobs_without_some_outputs():
    t = torch()
    x = Lp(5, 3000, "f32", 0, seed=4)
    lse = t.empty(5, device="cuda")
    fs.check(fs.fs_logprobs(x.p, x.logits, None, None, None, 0, None, None, lse, None, None, None, x.ws()))
    assert np.abs(f64(lse) - x.want["lse"]).max() < 1e-4
    rank = t.empty(5, dtype=t.int32, device="cuda")
    fs.check(fs.fs_logprobs(x.p, x.logits, None, None, x.token, 0, None, rank, None, None, None, None, x.ws()))
    assert np.array_equal(host(rank), x.want["rank"])
    # no vocabulary at all
    p = fs.params(3, 0, 0)
    o = Lp(3, 1, n_top=2).out()
    fs.check(fs.fs_logprobs(p, None, None, None, x.token[:3], 2, o["logprob"], o["rank"], o["lse"], o["entropy"],
                            o["top_idx"], o["top_logprob"], garbage(fs.fs_workspace_bytes(p, fs.FS_VARIANT_LOGPROBS, 2)),
                            dtype=fs.FS_F32))
    assert np.all(host(o["lse"]) == -np.inf) and np.all(host(o["logprob"]) == -np.inf)
    assert np.all(host(o["top_idx"]) == -1) and np.all(host(o["rank"]) == 0) and np.all(host(o["entropy"]) == 0)


def test_logprobs_workspace_is_checked():
    x = Lp(4, 151936, n_top=20)
    o = x.out()
    n = fs.fs_workspace_bytes(x.p, fs.FS_VARIANT_LOGPROBS, 20)
    a = (x.p, x.logits, None, None, x.token, 20, o["logprob"], o["rank"], o["lse"], o["entropy"], o["top_idx"],
         o["top_logprob"])
    assert fs.fs_logprobs(*a, None) == fs.FS_ERR_WORKSPACE
    assert fs.fs_logprobs(*a, x.ws(), n - 1) == fs.FS_ERR_WORKSPACE
    torch().cuda.synchronize()
    assert np.all(host(o["rank"]) == -7)


def test_logprobs_offsets_past_32_bits():
    """2.3e9 logits: the last rows lie behind 2^31 elements (and 2^32 bytes)."""
    t = torch()
    B, V, n = 15200, 151936, 3
    big = t.zeros((B, V), dtype=t.bfloat16, device="cuda")
    x = Lp(3, V, "bf16", n, seed=8)
    big[-3:] = x.logits
    tok = t.zeros(B, dtype=t.int32, device="cuda")
    tok[-3:] = x.token
    p = fs.params(B, 0, V)
    f, i = dict(dtype=t.float32, device="cuda"), dict(dtype=t.int32, device="cuda")
    o = dict(logprob=t.empty(B, **f), rank=t.empty(B, **i), lse=t.empty(B, **f), entropy=t.empty(B, **f),
             top_idx=t.empty((B, n), **i), top_logprob=t.empty((B, n), **f))
    ws = garbage(fs.fs_workspace_bytes(p, fs.FS_VARIANT_LOGPROBS, n))
    fs.check(fs.fs_logprobs(p, big, None, None, tok, n, o["logprob"], o["rank"], o["lse"], o["entropy"], o["top_idx"],
                            o["top_logprob"], ws))
    t.cuda.synchronize()
    x.check({k: v[-3:] for k, v in o.items()})
    assert bool((o["rank"][:-3] == 1).all()) and bool((o["top_idx"][:-3] == t.arange(3, device="cuda")).all())
    assert np.abs(f64(o["lse"][:-3]) - np.log(V)).max() < 2e-5
    # and their gradient, in place
    one = t.ones(B, **f)
    fs.check(fs.fs_logprobs_grad(p, big, None, None, tok, 0, None, o["lse"], None, one, None, None, None, big))
    t.cuda.synchronize()
    want, mag = OV.logprobs_grad(x.l, x.T, x.token_h, None, f64(o["lse"][-3:]), None, np.ones(3), None, None, None)
    check_grad(big[-3:], want, mag, "bf16")
    assert np.abs(f64(big[0, 1:100]) + 1 / V).max() <= 2.0 ** -8 / V


# ---------------------------------------------------------------------------
# their gradient
# ---------------------------------------------------------------------------
def check_grad(got, want, mag, dtype):
    """mag: the terms times the rounding steps each goes through."""
    err = np.abs(f64(got) - want)
    tol = HALF[dtype] * np.abs(want) + 4 * U * mag + TINY[dtype]
    assert np.all(err <= tol), (err - tol).max()


def grads(x, rng, which):
    g = {k: (rng.normal(size=x.B).astype(np.float32) if k in which else None) for k in ("lp", "lse", "ent")}
    g["top"] = rng.normal(size=(x.B, x.n_top)).astype(np.float32) if "top" in which and x.n_top else None
    return g


def run_grad(x, g, out=None, logits=None, stream=None):
    t = torch()
    lse, ent = dev(x.want["lse"].astype(np.float32)), dev(x.want["entropy"].astype(np.float32))
    idx = dev(x.want["top_idx"].astype(np.int32))
    out = t.full((x.B, x.V), 7.0, dtype=tdt(x.dtype), device="cuda") if out is None else out
    d = {k: None if v is None else dev(v) for k, v in g.items()}
    fs.check(fs.fs_logprobs_grad(x.p, x.logits if logits is None else logits, x.temp, x.allow, x.token, x.n_top, idx, lse,
                                 ent, d["lp"], d["lse"], d["ent"], d["top"], out, stream=stream), "fs_logprobs_grad")
    t.cuda.synchronize()
    return out


def want_grad(x, g):
    return OV.logprobs_grad(x.l, x.T, x.token_h, x.want["top_idx"], x.want["lse"].astype(np.float32).astype(np.float64),
                            x.want["entropy"].astype(np.float32).astype(np.float64), g["lp"], g["lse"], g["ent"], g["top"],
                            x.v_offset)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,V,n_top,pad,which", [
    (1, 1, 0, 0, ("lp",)), (3, 7, 3, 2, ("lp", "lse", "ent", "top")), (5, 1000, 0, 0, ("ent",)),
    (4, 4097, 64, 1, ("lp", "top")), (2, 50257, 8, 0, ("lp", "lse", "ent", "top")), (130, 515, 2, 9, ("lse", "top")),
    (33, 32000, 5, 0, ("lp", "ent"))])
def test_gradient_matches_the_oracle(B, V, n_top, pad, which, dtype):
    rng = np.random.default_rng(V)
    log(f"logprobs_grad B={B} V={V} n_top={n_top} pad={pad} {dtype} {which}")
    x = Lp(B, V, dtype, n_top, pad, temp=rng.uniform(0.4, 1.6, B) if B > 1 else None, seed=B,
           allow=some_mask(B, V, 4) if B % 2 else None)
    g = grads(x, rng, which)
    want, mag = want_grad(x, g)
    check_grad(run_grad(x, g), want, mag, dtype)
    # in place, and into rows that are further apart, where the gaps stay as they were
    buf = torch().full((B, V + 3), 5.0, dtype=tdt(dtype), device="cuda")
    check_grad(run_grad(x, g, buf[:, :V]), want, mag, dtype)
    assert bool((buf[:, V:] == 5.0).all())
    check_grad(run_grad(x, g, x.logits), want, mag, dtype)


def test_gradient_of_shards_masks_and_empty_rows():
    rng = np.random.default_rng(1)
    B, V = 6, 3001
    allow = some_mask(B, V, 9)
    allow[2] = 0
    token = np.array([48, -1, 50, 47, 48 + V, 48 + V - 1])
    x = Lp(B, V, "f32", 6, 2, np.array([1, 0.5, 1, 0, 2, -3]), allow, n_valid=48 + 2990, v_offset=48, token=token, seed=2)
    x.want["top_idx"][0, 1] = -1                   # an absent alternative
    x.want["top_idx"][1, 2] = 3                    # one of another shard
    x.want["top_idx"][3, 0] = x.want["top_idx"][3, 1]   # the same id twice: both gradients arrive
    g = grads(x, rng, ("lp", "lse", "ent", "top"))
    want, mag = want_grad(x, g)
    got = run_grad(x, g)
    check_grad(got, want, mag, "f32")
    assert np.all(host(got)[2] == 0) and np.all(host(got)[:, 2990:] == 0)


def test_gradient_follows_differences_of_the_forward_pass():
    """Central differences of the GPU's own forward pass, in float32: the
    step 2^-6 leaves h^2 / 6 of the third derivative (below 1e-4 here) and
    2 * 1e-5 / h of the values' rounding."""
    t = torch()
    rng = np.random.default_rng(7)
    B, V = 2, 60
    x = Lp(B, V, "f32", 0, temp=[0.8, 1.0], seed=1, std=1.5)
    g = grads(x, rng, ("lp", "lse", "ent"))
    got = f64(run_grad(x, g))

    def total():
        o = x.run()
        return sum((g[k].astype(np.float64) * f64(o[n])) for k, n in (("lp", "logprob"), ("lse", "lse"), ("ent", "entropy")))

    h = 2.0 ** -6
    for i in range(0, V, 7):
        keep = x.logits[:, i].clone()
        x.logits[:, i] = keep + h
        up = total()
        x.logits[:, i] = keep - h
        dn = total()
        x.logits[:, i] = keep
        assert np.abs((up - dn) / (2 * h) - got[:, i]).max() < 3e-3
    t.cuda.synchronize()


# ---------------------------------------------------------------------------
# embedding and its gradient
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,d,V", [(1, 1, 1), (1, 2048, 77), (5, 3, 10), (33, 256, 64), (257, 514, 100), (100, 4096, 50),
                                   (3, 5121, 9), (2000, 24, 300)])
def test_embed_matches_the_oracle(N, d, V, dtype):
    t = torch()
    rng = np.random.default_rng(N + d)
    W, Wf = as_type(rng.normal(size=(V, d)), dtype)
    ids = rng.integers(-2, V + 3, N) + 32          # a few lie outside
    scale = 11.313708
    out = t.full((N + 1, d), 7.0, dtype=tdt(dtype), device="cuda")
    log(f"embed N={N} d={d} V={V} {dtype}")
    fs.check(fs.fs_embed(fs.params(N, d, V, v_offset=32), dev(ids.astype(np.int32)), W, scale, out[:N]), "fs_embed")
    t.cuda.synchronize()
    want = OV.embed(ids, Wf, float(np.float32(scale)), 32)
    # one product in FP32, one rounding to the type
    assert np.all(np.abs(f64(out[:N]) - want) <= (HALF[dtype] + 2 * U) * np.abs(want) + TINY[dtype])
    assert bool((out[N] == 7.0).all())


def test_embed_shapes_at_the_edges():
    t = torch()
    out = t.full((3, 8), 7.0, device="cuda")
    ids = dev(np.array([0, -1, 2 ** 31 - 1], np.int32))
    fs.check(fs.fs_embed(fs.params(3, 8, 0), ids, None, 1.0, out, dtype=fs.FS_F32))
    assert bool((out == 0).all())
    # rows that start off 16 bytes
    W, Wf = as_type(np.random.default_rng(0).normal(size=(6, 8)), "bf16")
    buf = t.zeros(6 * 8 + 3, dtype=t.bfloat16, device="cuda")
    buf[3:] = W.flatten()
    o = t.full((3 * 8 + 1,), 7.0, dtype=t.bfloat16, device="cuda")
    fs.check(fs.fs_embed(fs.params(3, 8, 6), dev(np.array([5, 0, 3], np.int32)), buf[3:], 1.0, o[1:]))
    assert np.array_equal(f64(o[1:]).reshape(3, 8), Wf[[5, 0, 3]]) and float(o[0]) == 7.0


def test_embed_offsets_past_32_bits():
    t = torch()
    V, d = 600_000, 4096
    W = t.zeros((V, d), dtype=t.float16, device="cuda")
    W[-1] = t.arange(d, device="cuda")
    ids = t.arange(V, dtype=t.int32, device="cuda").flip(0).contiguous()
    out = t.full((V, d), 7.0, dtype=t.float16, device="cuda")
    fs.check(fs.fs_embed(fs.params(V, d, V), ids, W, 0.5, out))
    assert bool((out[0] == W[-1] * 0.5).all()) and bool((out[1:] == 0).all())
    W[0] = 1.0
    fs.check(fs.fs_embed(fs.params(V, d, V), ids, W, 0.5, out))
    assert bool((out[-1] == 0.5).all())
    # the gradient: dW behind 2^31 elements, and g too
    ws = garbage(fs.fs_workspace_bytes(fs.params(V, d, V), fs.FS_VARIANT_EMBED_GRAD))
    fs.check(fs.fs_embed_grad(fs.params(V, d, V), ids, out, 2.0, 0, W, ws))
    assert bool((W == out.flip(0) * 2).all())


def eg(ids, g, scale, V, out, accumulate=0, v_offset=0, stream=None, ws=None):
    N, d = g.shape
    p = fs.params(N, d, V, v_offset=v_offset)
    ws = garbage(fs.fs_workspace_bytes(p, fs.FS_VARIANT_EMBED_GRAD)) if ws is None else ws
    fs.check(fs.fs_embed_grad(p, ids, g, scale, accumulate, out, ws, stream=stream), "fs_embed_grad")
    return ws


def id_lists(V, N, kind, rng):
    if kind == "any":
        return rng.integers(-1, V + 2, N)
    if kind == "same":
        return np.full(N, V - 1)
    if kind == "two":
        return rng.choice([0, V - 1], N)
    if kind == "none":
        return rng.choice([-1, V, 2 ** 31 - 1, -2 ** 31], N)
    if kind == "zipf":
        return np.minimum((V ** rng.random(N)).astype(np.int64) - 1, V - 1)
    return np.arange(N)[::-1] % V                  # descending


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("N,d,V,kind", [
    (0, 8, 5, "any"), (1, 1, 1, "any"), (3, 5, 2, "any"), (64, 24, 10, "any"), (333, 256, 4096, "zipf"),
    (1000, 40, 7, "same"), (1025, 8, 50257, "any"), (4096, 16, 300, "two"), (70, 514, 40, "none"),
    (5000, 8, 4999, "down"), (9000, 32, 151936, "zipf"), (20000, 8, 1000, "zipf"), (257, 5121, 9, "any")])
def test_embed_gradient_matches_the_oracle(N, d, V, kind, dtype, out):
    t = torch()
    rng = np.random.default_rng(N + d)
    ids = id_lists(V, N, kind, rng)
    g, gf = as_type(rng.normal(size=(N, d)), dtype)
    scale = 1.75
    log(f"embed_grad N={N} d={d} V={V} {kind} {dtype} -> {out}")
    want, mag = OV.embed_grad(ids, gf, scale, V)
    count = np.bincount(ids[(ids >= 0) & (ids < V)], minlength=V)[:, None]
    # a sum of n terms: n roundings at most, one more for the scale, one for the type
    tol = HALF[out] * np.abs(want) + U * (count + 2) * mag + TINY[out]
    ids_d = dev(np.asarray(ids, np.int64).astype(np.int32))
    dW = t.full((V + 1, d), 7.0, dtype=tdt(out), device="cuda")
    eg(ids_d, g, scale, V, dW[:V])
    err = np.abs(f64(dW[:V]) - want)
    assert np.all(err <= tol), (err - tol).max()
    assert np.all(f64(dW[:V])[count[:, 0] == 0] == 0) and bool((dW[V] == 7.0).all())
    # added to what is there; rows without an id are not touched
    base, basef = as_type(rng.normal(size=(V, d)), out)
    acc = base.clone()
    eg(ids_d, g, scale, V, acc, accumulate=1)
    err = np.abs(f64(acc) - (want + basef))
    assert np.all(err <= tol + HALF[out] * np.abs(want + basef) + U * np.abs(basef))
    assert np.array_equal(f64(acc)[count[:, 0] == 0], basef[count[:, 0] == 0])


@pytest.mark.parametrize("kind,dtype,out", [("zipf", "bf16", "bf16"), ("two", "f32", "f32"), ("any", "f16", "f32")])
def test_embed_gradient_of_long_lists(kind, dtype, out):
    test_embed_gradient_matches_the_oracle(17000, 1001, 300, kind, dtype, out)   # (chunks of 32)


def test_embed_gradient_is_the_same_every_time():
    t = torch()
    rng = np.random.default_rng(2)
    N, d, V = 6000, 264, 500
    ids = dev(id_lists(V, N, "zipf", rng).astype(np.int32))
    g, _ = as_type(rng.normal(size=(N, d)), "bf16")
    first = None
    for i in range(4):
        dW = t.full((V, d), float(i), device="cuda")
        eg(ids, g, 1.0, V, dW)
        first = dW if first is None else first
        assert bool((dW == first).all())


def test_embed_gradient_of_a_shard():
    t = torch()
    rng = np.random.default_rng(4)
    N, d, V, off = 700, 48, 90, 64
    ids = rng.integers(0, 300, N)
    g, gf = as_type(rng.normal(size=(N, d)), "f32")
    dW = t.empty((V, d), device="cuda")
    eg(dev(ids.astype(np.int32)), g, 1.0, V, dW, v_offset=off)
    want, mag = OV.embed_grad(ids, gf, 1.0, V, off)
    assert np.all(np.abs(f64(dW) - want) <= 64 * U * mag)
    # off 16 bytes, and the workspace's size is checked
    buf, ob = t.zeros(N * d + 1, device="cuda"), t.full((V * d + 3,), 7.0, device="cuda")
    buf[1:] = g.flatten()
    eg(dev(ids.astype(np.int32)), buf[1:].view(N, d), 1.0, V, ob[3:].view(V, d), v_offset=off)
    assert bool((ob[3:].view(V, d) == dW).all()) and bool((ob[:3] == 7.0).all())
    p = fs.params(N, d, V)
    n = fs.fs_workspace_bytes(p, fs.FS_VARIANT_EMBED_GRAD)
    assert fs.fs_embed_grad(p, dev(ids.astype(np.int32)), g, 1.0, 0, dW, None) == fs.FS_ERR_WORKSPACE
    assert fs.fs_embed_grad(p, dev(ids.astype(np.int32)), g, 1.0, 0, dW, garbage(n), n - 1) == fs.FS_ERR_WORKSPACE


# ---------------------------------------------------------------------------
# together, on streams and in graphs
# ---------------------------------------------------------------------------
def test_tensors_that_do_not_fit_are_refused():
    t = torch()
    z = lambda *s, **k: t.zeros(s, device="cuda", **k)  # noqa: E731
    p, ids, BAD = fs.params(2, 8, 4), z(2, dtype=t.int32), fs.FS_ERR_INVALID_ARG
    ok = (z(2), None, None, None, None, None, z(1024, dtype=t.uint8))
    assert fs.fs_logprobs(p, z(2, 4), None, None, ids, 0, *ok) == fs.FS_OK
    assert fs.fs_logprobs(p, z(2, 8)[:, ::2], None, None, ids, 0, *ok) == BAD
    assert fs.fs_logprobs(p, z(3, 4), None, None, ids, 0, *ok) == BAD
    assert fs.fs_logprobs(p, z(2, 4, dtype=t.float64), None, None, ids, 0, *ok) == BAD
    assert fs.fs_logprobs(p, t.zeros(2, 4), None, None, ids, 0, *ok) == BAD
    assert fs.fs_logprobs(p, z(2, 4), None, None, z(4, dtype=t.int32)[::2], 0, *ok) == BAD
    assert fs.fs_embed(p, ids, z(4, 8), 1.0, z(2, 8)) == fs.FS_OK
    assert fs.fs_embed(p, ids, z(8, 4).T, 1.0, z(2, 8)) == BAD
    assert fs.fs_embed(p, ids, z(4, 8), 1.0, z(2, 8, dtype=t.float16)) == BAD
    assert fs.fs_embed(p, ids, z(4, 8), 1.0, t.zeros(2, 8)) == BAD
    assert fs.fs_embed_grad(p, ids, z(8, 2).T, 1.0, 0, z(4, 8), z(1 << 16, dtype=t.uint8)) == BAD
    t.cuda.synchronize()


def test_tensors_of_another_type_are_refused():
    t = torch()
    z = lambda *s, **k: t.zeros(s, device="cuda", **k)  # noqa: E731
    p, BAD = fs.params(2, 64, 4), fs.FS_ERR_INVALID_ARG
    ids, long = z(2, dtype=t.int32), z(2, dtype=t.int64)
    ws = z(1 << 16, dtype=t.uint8)
    l, row = z(2, 4), z(2)
    idx, val = z(2, 1, dtype=t.int32), z(2, 1)
    call = lambda temp=None, allow=None, tok=ids, lp=row, rank=None, idx=idx, val=val: fs.fs_logprobs(  # noqa: E731
        p, l, temp, allow, tok, 1, lp, rank, None, None, idx, val, ws)
    assert call() == call(temp=row, allow=z(2, 1, dtype=t.int32), rank=ids) == fs.FS_OK
    for bad in (dict(temp=row.double()), dict(allow=z(2, 1, dtype=t.int64)), dict(tok=long), dict(lp=row.half()),
                dict(rank=long), dict(idx=idx.long()), dict(val=val.double())):
        assert call(**bad) == BAD, bad
    grad = lambda lse=row, tok=ids, g=row: fs.fs_logprobs_grad(  # noqa: E731
        p, l, None, None, tok, 0, None, lse, None, g, None, None, None, z(2, 4))
    assert grad() == fs.FS_OK
    assert grad(lse=row.double()) == grad(tok=long) == grad(g=row.bfloat16()) == BAD
    W, out = z(4, 64), z(2, 64)
    assert fs.fs_embed(p, ids, W, 1.0, out) == fs.FS_OK
    assert fs.fs_embed(p, long, W, 1.0, out) == BAD
    assert fs.fs_embed_grad(p, ids, out, 1.0, 0, W, ws) == fs.FS_OK
    assert fs.fs_embed_grad(p, long, out, 1.0, 0, W, ws) == BAD
    q, s = z(4, 32, dtype=t.uint8), z(4, 2, dtype=t.bfloat16)
    H = z(2, 64, dtype=t.bfloat16)
    assert fs.fs_logits_quant(p, H, fs.quant(q, s, None, 32), l) == fs.FS_OK
    assert fs.fs_logits_quant(p, H.half(), fs.quant(q, s, None, 32), l) == BAD
    assert fs.fs_logits_quant(p, H, fs.quant(q, s, None, 32), l.bfloat16()) == BAD
    for args in ((q.int(), s, None), (q, s, s)):
        with pytest.raises(ValueError):
            fs.quant(*args, 32)
    t.cuda.synchronize()


def test_more_rows_than_a_grid_has():
    # each workgroup takes a second row: rows repeat with a period of 997
    t = torch()
    B, V, per = 66001, 70, 997
    x = Lp(per, V, "f32", 3, seed=5)
    g = grads(x, np.random.default_rng(6), ("lp", "lse", "ent", "top"))
    want, mag = want_grad(x, g)
    at = t.arange(B, device="cuda") % per
    big = lambda v: v.index_select(0, at) if hasattr(v, "shape") else v  # noqa: E731
    p, ws = fs.params(B, 0, V), garbage(fs.fs_workspace_bytes(fs.params(B, 0, V), fs.FS_VARIANT_LOGPROBS, 3))
    o = {k: big(v) for k, v in x.out().items()}
    logits, token = big(x.logits), big(x.token)
    fs.check(fs.fs_logprobs(p, logits, None, None, token, 3, o["logprob"], o["rank"], o["lse"], o["entropy"], o["top_idx"],
                            o["top_logprob"], ws))
    out = t.empty_like(logits)
    d = {k: big(dev(v)) for k, v in g.items()}
    fs.check(fs.fs_logprobs_grad(p, logits, None, None, token, 3, big(dev(x.want["top_idx"].astype(np.int32))),
                                 big(dev(x.want["lse"].astype(np.float32))), big(dev(x.want["entropy"].astype(np.float32))),
                                 d["lp"], d["lse"], d["ent"], d["top"], out))
    t.cuda.synchronize()
    x.check({k: v[:per] for k, v in o.items()})
    check_grad(out[:per], want, mag, "f32")
    for v in (*o.values(), out):
        assert bool((v == big(v[:per])).all())


def decode_state(seed):
    """One decode step around a 4-bit head: embed the last tokens, logits,
    draw, and the log probability of the draw with alternatives."""
    t = torch()
    B, d, V, group, n = 6, 256, 5003, 64, 5
    H, Hf, q, S, Sf, z = quant_problem(B, d, V, group, "bf16", True, seed=seed)
    rng = np.random.default_rng(seed + 100)
    E, Ef = as_type(rng.normal(size=(V, d)), "bf16")
    s = dict(B=B, d=d, V=V, n=n, group=group, q=q, Sf=Sf, z=z, Ef=Ef, E=E, S=S, keep=(dev(q), dev(z)))
    s["W"] = fs.quant(s["keep"][0], S, s["keep"][1], group)
    s["step"] = t.zeros(1, dtype=t.int32, device="cuda")
    s["p"] = fs.params(B, d, V, seed=17, step_ptr=s["step"])
    s["ids"] = dev(np.arange(B, dtype=np.int32))
    s["H"] = t.empty((B, d), dtype=t.bfloat16, device="cuda")
    s["logits"] = t.empty((B, V), device="cuda")
    s["ws"] = garbage(fs.fs_workspace_bytes(s["p"], fs.FS_VARIANT_LOGPROBS, n))
    s["mws"] = garbage(fs.fs_workspace_bytes(s["p"], fs.FS_VARIANT_MULTINOMIAL))
    s["lp"] = t.empty(B, device="cuda")
    s["rank"] = t.empty(B, dtype=t.int32, device="cuda")
    s["top"] = t.empty((B, n), dtype=t.int32, device="cuda")
    s["top_lp"] = t.empty((B, n), device="cuda")
    return s


def decode_step(s, stream=None):
    fs.check(fs.fs_embed(s["p"], s["ids"], s["E"], 1.0, s["H"], stream=stream))
    fs.check(fs.fs_logits_quant(s["p"], s["H"], s["W"], s["logits"], stream=stream))
    fs.check(fs.fs_multinomial(s["p"], s["logits"], None, None, s["ids"], s["mws"], stream=stream))
    fs.check(fs.fs_logprobs(s["p"], s["logits"], None, None, s["ids"], s["n"], s["lp"], s["rank"], None, None, s["top"],
                            s["top_lp"], s["ws"], stream=stream))


def decode_check(s, last):
    """One step against the oracle, from the ids that went in."""
    Hf = OV.embed(last, s["Ef"], 1.0)
    want = Hf @ OV.dequantise(s["q"], s["Sf"], s["z"], s["group"]).T
    assert np.all(np.abs(f64(s["logits"]) - want) <= quant_bound(Hf, s["q"], s["Sf"], s["z"], s["group"]))
    ids = host(s["ids"])
    assert np.all((ids >= 0) & (ids < s["V"]))
    r = OV.logprobs(f64(s["logits"]), np.ones(s["B"]), ids, s["n"])
    assert np.array_equal(host(s["rank"]), r["rank"]) and np.array_equal(host(s["top"]), r["top_idx"])
    near(s["lp"], r["logprob"], 400 * U * (1 + np.abs(r["logprob"])))


def test_decode_loop_eager_and_captured():
    t = torch()
    s = decode_state(1)
    seen = []
    for i in range(4):
        last = host(s["ids"]).copy()
        decode_step(s)
        s["step"].add_(1)
        t.cuda.synchronize()
        decode_check(s, last)
        seen.append((host(s["ids"]).copy(), host(s["lp"]).copy()))
    # the same loop from a graph, with eager work between the replays
    c, other = decode_state(1), decode_state(2)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        decode_step(c)
    t.cuda.current_stream().wait_stream(side)
    c["ids"].copy_(dev(np.arange(c["B"], dtype=np.int32)))
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        decode_step(c)
        c["step"].add_(1)
    for i in range(4):
        last = host(c["ids"]).copy()
        graph.replay()
        decode_step(other)                         # an eager step of another state right behind it
        t.cuda.synchronize()
        decode_check(c, last)
        assert np.array_equal(host(c["ids"]), seen[i][0]) and np.array_equal(host(c["lp"]), seen[i][1])


def train_step(s, stream=None):
    """Scores of given tokens under a tied head, and the gradient of the table
    from both ends."""
    t = torch()
    fs.check(fs.fs_embed(s["p"], s["ids"], s["W"], 2.0, s["H"], stream=stream))
    fs.check(fs.fs_logits(s["p"], s["H"], s["W"], s["logits"], s["lws"], stream=stream))
    fs.check(fs.fs_logprobs(s["p"], s["logits"], None, None, s["token"], 0, s["lp"], None, s["lse"], s["ent"], ws=s["ws"],
                            stream=stream))
    fs.check(fs.fs_logprobs_grad(s["p"], s["logits"], None, None, s["token"], 0, None, s["lse"], s["ent"], s["g"], None,
                                 s["ge"], None, s["logits"], stream=stream))
    with t.cuda.stream(stream or t.cuda.current_stream()):
        s["dH"].copy_(s["logits"] @ s["W"].float())
        s["dW"].copy_(s["logits"].t() @ s["H"].float())
    fs.check(fs.fs_embed_grad(s["p"], s["ids"], s["dH"], 2.0, 1, s["dW"], s["ews"], stream=stream))


def train_state(seed):
    t = torch()
    rng = np.random.default_rng(seed)
    N, d, V = 48, 64, 1600
    s = dict(N=N, d=d, V=V)
    s["W"], s["Wf"] = as_type(0.3 * rng.normal(size=(V, d)), "bf16")
    s["ids_h"], s["tok_h"] = id_lists(V, N, "zipf", rng), rng.integers(0, V, N)
    s["ids"], s["token"] = dev(s["ids_h"].astype(np.int32)), dev(s["tok_h"].astype(np.int32))
    s["g_h"], s["ge_h"] = rng.normal(size=N).astype(np.float32), 0.1 * rng.normal(size=N).astype(np.float32)
    s["g"], s["ge"] = dev(s["g_h"]), dev(s["ge_h"].astype(np.float32))
    s["p"] = fs.params(N, d, V)
    s["H"] = t.empty((N, d), dtype=t.bfloat16, device="cuda")
    for k, shape in (("logits", (N, V)), ("lp", (N,)), ("lse", (N,)), ("ent", (N,)), ("dH", (N, d)), ("dW", (V, d))):
        s[k] = t.empty(shape, device="cuda")
    s["lws"] = garbage(fs.fs_workspace_bytes(s["p"], fs.FS_VARIANT_LOGITS))
    s["ws"] = garbage(fs.fs_workspace_bytes(s["p"], fs.FS_VARIANT_LOGPROBS, 0))
    s["ews"] = garbage(fs.fs_workspace_bytes(s["p"], fs.FS_VARIANT_EMBED_GRAD))
    return s


def test_training_step_on_streams_and_in_a_graph():
    """The tied table's gradient against float64; the same bits from two
    streams at once and from replays of a graph."""
    t = torch()
    s = train_state(3)
    train_step(s)
    t.cuda.synchronize()
    Hf = f64(s["H"])
    l = Hf @ s["Wf"].T
    r = OV.logprobs(l, np.ones(s["N"]), s["tok_h"], 0)
    dl, _ = OV.logprobs_grad(l, np.ones(s["N"]), s["tok_h"], None, r["lse"], r["entropy"], s["g_h"], None,
                             s["ge_h"], None)
    dW = dl.T @ Hf + OV.embed_grad(s["ids_h"], dl @ s["Wf"], 2.0, s["V"])[0]
    # FP32 all the way after H: sums of N and V terms, each off by a few hundred u of the largest
    assert np.abs(f64(s["dW"]) - dW).max() <= 4000 * U * np.abs(dW).max()
    assert np.abs(f64(s["lp"]) - r["logprob"]).max() <= 1000 * U * (1 + np.abs(l).max())
    a, b = train_state(3), train_state(4)
    train_step(b)
    t.cuda.synchronize()
    ref_b = b["dW"].clone()
    b["dW"].zero_()
    s1, s2 = t.cuda.Stream(), t.cuda.Stream()
    t.cuda.synchronize()
    for _ in range(3):
        train_step(a, s1)
        train_step(b, s2)
    t.cuda.synchronize()
    assert bool((a["lp"] == s["lp"]).all()) and bool((a["lse"] == s["lse"]).all())
    scale = float(s["dW"].abs().max())
    assert float((a["dW"] - s["dW"]).abs().max()) <= 100 * U * scale    # the library products may differ by stream
    assert float((b["dW"] - ref_b).abs().max()) <= 100 * U * float(ref_b.abs().max())
    # captured: the framework's calls alone
    c = train_state(3)
    c["logits"].copy_(s["logits"])
    dH = s["dH"].clone()

    def calls():
        fs.check(fs.fs_embed(c["p"], c["ids"], c["W"], 2.0, c["H"]))
        fs.check(fs.fs_logits(c["p"], c["H"], c["W"], c["logits"], c["lws"]))
        fs.check(fs.fs_logprobs(c["p"], c["logits"], None, None, c["token"], 0, c["lp"], None, c["lse"], c["ent"],
                                ws=c["ws"]))
        fs.check(fs.fs_logprobs_grad(c["p"], c["logits"], None, None, c["token"], 0, None, c["lse"], c["ent"], c["g"],
                                     None, c["ge"], None, c["logits"]))
        fs.check(fs.fs_embed_grad(c["p"], c["ids"], dH, 2.0, 0, c["dW"], c["ews"]))

    calls()
    t.cuda.synchronize()
    ref = {k: c[k].clone() for k in ("lp", "lse", "ent", "logits", "dW")}
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        calls()
    for i in range(4):
        for k in ("lp", "lse", "ent", "logits", "dW"):
            c[k].fill_(float(i))
        graph.replay()
        train_step(b)
        t.cuda.synchronize()
        for k, v in ref.items():
            assert bool((c[k] == v).all()), (i, k)
