"""Every launch form of the attention half that sizes choose, each with the check that the call took it: the names of the kernels
that a captured call holds."""
import ctypes
import re

import numpy as np
import pytest
import torch

import attn_reference as ref
import test_gpu_attn as base
from block_scaled_fp4_moe_gb300 import _build, attn, moe

pytestmark = pytest.mark.gpu
built = base.built


def kernels(call, tmp_path):
    """The kernel names, as the linker has them, of what `call` launches."""
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    path = tmp_path / "graph.dot"
    assert ctypes.CDLL("libcuda.so.1").cuGraphDebugDotPrint(ctypes.c_void_p(g.raw_cuda_graph()), str(path).encode(), 0) == 0
    return re.findall(r"_Z\w*_kernel\w*", path.read_text())


def has(names, kernel, *args):
    """One of them is the kernel with these template arguments (whole numbers and truth values)."""
    coded = "".join(f"Lb{int(a)}E" if isinstance(a, bool) else f"Li{a}E" for a in args)
    return any(kernel + (f"I{coded}E" if args else "") in n for n in names)


# --------------------------------------------------------------- attention

class Recorded(base.Problem):
    """A problem whose call is captured for its kernels' names as well."""

    def kernels(self, tmp_path, causal=True, window=0):
        dev = attn.KVCache(*[torch.from_numpy(a).cuda() for a in self.cache.layout()])
        heads = self.q.shape[1]
        out = torch.empty(self.q.shape, dtype=torch.bfloat16, device="cuda")
        ws = base.workspace(attn.moe_kv_attention_workspace_size(self.T, len(self.kv), heads, dev.kv_heads, self.dim))
        args = [self.q, dev, base.i32(self.table), base.i32(self.offsets), base.i32(self.kv), self.scale, out, None, ws]
        return kernels(lambda: attn.moe_kv_attention(*args, causal=causal, window=window), tmp_path)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("B,new,kv_heads,group", [(300, 1, 2, 4), (256, 6, 1, 4), (1100, 1, 1, 2), (2500, 1, 1, 2)])
def test_attention_with_a_plan_made_beforehand(dim, B, new, kv_heads, group, tmp_path):
    """More than 256 requests, or more than 288 row tiles; more than 1,024 requests: a plan of several passes over them."""
    rng = np.random.default_rng(B + dim)
    lens = [(int(rng.integers(0, new + 1)), int(k)) for k in rng.integers(0, 90, B)]
    lens[0], lens[-1], lens[B // 2] = (new, 700), (new, 1), (new, 0)
    p = Recorded(lens, kv_heads, group, dim, 16, seed=60)
    names = p.kernels(tmp_path)
    assert has(names, "attn_plan_kernel") and has(names, "attn_kernel", dim, False), names
    p.check()
    p.check(causal=False, window=20)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("B", [8, 300, 1100])
def test_attention_of_many_rows_and_requests(dim, B, tmp_path):
    rng = np.random.default_rng(B + dim)
    lens = [(int(n), int(k)) for n, k in zip(rng.integers(5, 9, B), rng.integers(0, 60, B))]
    lens[0], lens[-1] = (8, 500), (8, 3)
    p = Recorded(lens, 8 if B == 8 else 1, 4, dim, 32, seed=61)
    if B == 8:
        p = Recorded([(n + 4, k) for n, k in lens], 8, 4, dim, 32, seed=61)
    names = p.kernels(tmp_path)
    assert has(names, "attn_plan_kernel") and has(names, "attn_tc_kernel", dim), names
    p.check()


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_with_a_plan_in_shared_memory(dim, tmp_path):
    p = Recorded([(1, 300), (2, 40), (1, 1)] * 85, 1, 2, dim, 16, seed=62)
    names = p.kernels(tmp_path)
    assert has(names, "attn_kernel", dim, True) and len(names) == 1, names
    p.check()


# ------------------------------------------------------------------ append

def append_case(lens, starts, heads, dim, size, seed):
    """Runs of `lens` tokens from `starts` on into blocks that hold what was there, from strided views."""
    rng = np.random.default_rng(seed)
    need = [-(-(s + n) // size) for s, n in zip(starts, lens)]
    cache, g, mirror = base.new_cache(sum(need) + 2, heads, dim, size, rng)
    order, at, slots = rng.permutation(sum(need) + 2), 0, []
    for n, s, m in zip(lens, starts, need):
        ids = order[at: at + m]
        at += m
        slots += [int(ids[p // size]) * size + p % size for p in range(s, s + n)]
        if rng.random() < 0.3:
            slots.append(-1)                               # a token that is left out, behind a request's
    slots = np.array(slots)
    x = base.bf16(rng.standard_normal((len(slots), 2 * heads + 1, dim)) * np.exp2(rng.integers(-9, 10, (len(slots), 1, 1))))
    return cache, g, mirror, x[:, :heads], x[:, heads + 1:], slots


@pytest.mark.parametrize("dim,heads", [(64, 3), (128, 2)])
@pytest.mark.parametrize("size", [16, 32, 64, 128])
@pytest.mark.parametrize("kind", ["prompts", "mixed", "short"])
def test_append_of_more_tokens_than_1024(kind, size, dim, heads, tmp_path):
    """A CTA looks at 32 tokens: long runs that begin anywhere in a window and reach past it, several of them in one, short ones between;
    only long ones; only short ones."""
    rng = np.random.default_rng(size + dim)
    if kind == "prompts":
        lens = [700, 513, 129, 64]
    elif kind == "mixed":
        lens = [int(n) for n in np.where(rng.random(90) < 0.6, rng.integers(1, 5, 90), rng.integers(5, 60, 90))]
        lens += [400, 1, 1, 300]
    else:
        lens = [int(n) for n in rng.integers(1, 4, 700)]
    starts = [int(s) for s in rng.integers(0, 2 * size, len(lens))]
    cache, g, mirror, k, v, slots = append_case(lens, starts, heads, dim, size, seed=63)
    assert len(slots) > 1024
    ws = base.workspace(512)
    attn.moe_kv_append(k, v, torch.from_numpy(slots).cuda(), cache, ws)
    assert base.status(ws) == 0
    mirror.append(base.f64(k), base.f64(v), slots)
    base.check_cache(g, mirror, kind)


@pytest.mark.parametrize("T", [1023, 1024, 1025, 1057])
def test_append_at_the_change_of_windows(T):
    cache, g, mirror, k, v, slots = append_case([T], [5], 1, 64, 64, seed=64)
    slots, k, v = slots[:T], k[:T], v[:T]
    ws = base.workspace(512)
    attn.moe_kv_append(k, v, torch.from_numpy(slots).cuda(), cache, ws)
    assert base.status(ws) == 0
    mirror.append(base.f64(k), base.f64(v), slots)
    base.check_cache(g, mirror)


# -------------------------------------------------------------- projection

def check_linear(T, N, K, seed, tmp_path, *form):
    xt, _, weight, y = base.linear_case(T, N, K, seed=seed)
    ws = base.workspace(attn.moe_linear_fp8_workspace_size(T, N, K))
    again = torch.empty_like(y)
    names = kernels(lambda: attn.moe_linear_fp8(xt, weight, again, ws), tmp_path)
    assert has(names, "fp8_gemm_kernel", *form), names
    want, bound = ref.linear(base.f64(xt), weight.codes.cpu().numpy(), weight.scale.cpu().numpy())
    err = np.abs(base.f64(y) - want)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("T,N,K", [(1000, 10001, 1040), (700, 15007, 656), (1300, 5003, 4112), (150, 10000, 2064), (180, 12001, 528), (1000, 9001, 512)])
def test_linear_persistent_form_goes_round_its_ring_and_accumulators(T, N, K, tmp_path):
    """More stages than the ring holds, in one tile and over several; three and more tiles a CTA; odd ends of N, K and the tokens."""
    check_linear(T, N, K, T + N, tmp_path, 192, False, False)


@pytest.mark.parametrize("T,tile,fused", [(1, 16, True), (8, 16, True), (9, 16, False), (16, 16, False), (17, 32, False), (40, 64, False),
                                          (100, 128, False), (200, 128, False)])
@pytest.mark.parametrize("N,K", [(1001, 4112), (7003, 1040)])
def test_linear_split_forms_go_round_their_rings(T, tile, fused, N, K, tmp_path):
    check_linear(T, N, K, T, tmp_path, tile, True, fused)


# ------------------------------------------- the build with range checks

@pytest.fixture
def debug():
    _build.build(debug=True)
    with moe.debug_bounds():
        yield


@pytest.mark.parametrize("kv_heads,group,dim,lens", [
    (2, 4, 64, [(1, 700), (3, 200), (0, 5), (1, 1)]), (1, 8, 128, [(1, 9000)]), (2, 8, 128, [(4, 900), (3, 40)]), (2, 8, 64, [(8, 5000), (7, 30)]),
    (1, 2, 64, [(1, 1 + i % 140) for i in range(300)]), (8, 4, 64, [(9, 700), (20, 300), (40, 200), (8, 90)]),
    (8, 8, 128, [(40, 5000), (9, 300), (70, 260), (12, 130)]), (8, 4, 128, [(8, 9000)] + [(8, 150 + 70 * i) for i in range(9)])])
def test_attention_under_range_checks(kv_heads, group, dim, lens, debug):
    """Rows, parts of cut units and their tickets stay in their ranges, in every form."""
    base.Problem(lens, kv_heads, group, dim, 32, seed=67).check()
    base.Problem(lens, kv_heads, group, dim, 16, seed=68).check(window=150)


def test_a_step_under_range_checks(debug):
    base.test_step_against_the_reference()
    base.test_tables_match_the_definition(65, 32, 300, 40, 0)
    for T in (1, 40, 300):
        base.test_linear_token_counts(T)


@pytest.mark.parametrize("T,gap", [(40, 1), (40, 3), (40, 40), (40, 127), (1500, 1), (1500, 100)])
def test_append_that_goes_on_with_a_block_behind_skipped_tokens(T, gap, debug):
    """Two runs of one block would settle its scale beside one another, which slot_map must not ask for: the range-checked build leaves the
    second out, and reports it."""
    cache, g, mirror, k, v, slots = append_case([T + gap + 300], [0], 2, 64, 64, seed=65)
    k, v, slots = k[:len(slots)], v[:len(slots)], slots.copy()
    at = T // 64 * 64 + 7                                  # inside a block
    slots[at:at + gap] = -1
    end = (at // 64 + 1) * 64
    ws = base.workspace(512)
    attn.moe_kv_append(k, v, torch.from_numpy(slots).cuda(), cache, ws)
    late = at + gap < end                                  # something of the block is left behind the gap
    assert base.status(ws) == (moe.MOE_ERR_DEVICE_ASSERT if late else 0)
    if late:
        slots[at + gap:end] = -1
    mirror.append(base.f64(k), base.f64(v), slots)
    base.check_cache(g, mirror)


def test_append_that_jumps_inside_a_block_is_reported(debug):
    for slots in ([0, 2], [5, 4], [7, 7]):
        cache, g, mirror, k, v, _ = append_case([2], [0], 1, 64, 64, seed=66)
        ws = base.workspace(512)
        attn.moe_kv_append(k[:2], v[:2], torch.tensor(slots).cuda(), cache, ws)
        assert base.status(ws) == moe.MOE_ERR_DEVICE_ASSERT
        for x in g:
            x.check()
