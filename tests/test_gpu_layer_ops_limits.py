"""Norm, rotary positions, latent append and latent attention at the ends of what their calls take."""
import ctypes as C
import threading

import pytest
import torch

import layer_ops_reference as ref
from block_scaled_fp4_moe_gb300 import _build, attn, moe
from test_gpu_layer_ops import Guarded, Step, gen, i32, normal, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("inter", [False, True])
def test_latent_append_leaves_out_tokens_before_the_first_position(latent, inter):
    """As moe_rotary does: nothing is written, although their slots are in the cache."""
    g = gen(70 + latent)
    pos = [5, -1, 0, -(2 ** 31), 2 ** 31 - 1, -7, 1 << 20]
    T = len(pos)
    both = normal(g, T, latent + 64)
    data = Guarded((2, 16, latent + 64), torch.bfloat16)
    before, ws = data.t.clone(), torch.zeros(512, dtype=torch.uint8, device="cuda")
    slots = torch.randperm(32, generator=g, device="cuda")[:T].clone()
    table = attn.RotaryTable.make(64)
    attn.moe_latent_append(both[:, :latent], both[:, latent:], slots, attn.LatentCache(data.t), ws, positions=i32(pos), table=table, interleaved=inter)
    assert moe.moe_check_device_status(ws) == 0
    data.check()
    live = i32(pos) >= 0
    rows, kept = data.t.view(32, -1), before.view(32, -1)
    want, bound = ref.rotary(both[live][:, None, latent:], i32(pos)[live], table.turns, 1.0, inter)
    within(rows[slots[live]][:, latent:], want[:, 0], bound[:, 0], "key")
    assert torch.equal(rows[slots[live]][:, :latent], both[live][:, :latent])
    rest = torch.ones(32, dtype=torch.bool, device="cuda")
    rest[slots[live]] = False
    assert torch.equal(rows[rest].view(torch.int16), kept[rest].view(torch.int16))


def test_latent_attention_from_two_host_threads():
    """Each on a stream and a workspace of its own, with head counts whose kernels take different amounts of shared memory.  Through the C
    ABI, which holds no lock while it launches."""
    L = attn.lib()
    steps = [Step([300, 90], [1, 1], 64, 512, 64, seed=71), Step([300, 90], [1, 1], 16, 512, 64, seed=72)]
    want = [s.run() for s in steps]
    calls, keep = [], []
    for s in steps:
        T, H, out, ws = s.T, s.heads, torch.empty(s.T, s.heads, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(s.ws)
        offsets, lens, stream = i32(s.offsets), i32(s.kv), torch.cuda.Stream()
        cache = attn._LatentCache(s.data.data_ptr(), s.data.shape[0], 512, 64)
        keep.append((out, ws, offsets, lens, stream, cache))
        args = (s.ql.data_ptr(), s.ql.stride(0), s.ql.stride(1), s.qr.data_ptr(), s.qr.stride(0), s.qr.stride(1), T, H, C.byref(cache), s.table.data_ptr(),
                s.table.shape[1], offsets.data_ptr(), lens.data_ptr(), 2, s.scale, 1, out.data_ptr(), None, ws.data_ptr(), ws.numel(), stream.cuda_stream)
        calls.append(lambda args=args: L.moe_latent_attention(*args))
    torch.cuda.synchronize()
    statuses = [[], []]
    start = threading.Barrier(2)

    def go(i):
        torch.zeros(1, device="cuda")
        start.wait()
        for _ in range(4000):
            statuses[i].append(calls[i]())
    threads = [threading.Thread(target=go, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [{v: st.count(v) for v in set(st)} for st in statuses] == [{moe.MOE_OK: 4000}] * 2
    for k, (out, _) in zip(keep, want):
        assert torch.equal(k[0], out) and moe.moe_check_device_status(k[1]) == 0


@pytest.mark.parametrize("what", ["latent attention", "projection", "projection of few tokens", "attention", "norm", "rotary", "append"])
def test_a_call_as_the_first_that_a_host_thread_makes(what):
    """A thread that has no CUDA context yet, as a server's worker that is handed tensors and calls a step."""
    s = Step([300, 90], [1, 1], 16, 512, 64, seed=73)
    want, _ = s.run()
    g = gen(74)
    x, w = normal(g, 40 if what == "projection" else 2, 512), attn.FP8Weight.from_dense(normal(g, 256, 512))
    ws, norm = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda"), normal(g, 512)
    table, pos, slots = attn.RotaryTable.make(64), i32([3, 4]), torch.tensor([0, 1], device="cuda")
    kv = attn.KVCache.empty(8, 2, 64, 32)
    for t in (kv.k, kv.v, kv.k_scale, kv.v_scale):
        t.zero_()
    heads, block_table, kv_lens = normal(g, 2, 4, 64), i32([[0, 1], [2, 3]]), i32([40, 30])
    latent = attn.LatentCache(s.data)
    lens, offsets = i32(s.kv), i32(s.offsets)

    def call():
        out = torch.zeros_like(want) if what == "latent attention" else torch.zeros(x.shape[0], 256, dtype=torch.bfloat16, device="cuda") if "proj" in what \
            else torch.zeros_like(heads) if what in ("attention", "rotary") else torch.zeros(8, 32, 576, dtype=torch.bfloat16, device="cuda") if what == "append" \
            else torch.zeros_like(x)
        to = attn.LatentCache(out) if what == "append" else None
        stream = torch.cuda.current_stream()
        torch.cuda.synchronize()
        return out, {
            "latent attention": lambda: attn.moe_latent_attention(s.ql, s.qr, latent, s.table, offsets, lens, s.scale, out, None, ws, stream=stream),
            "attention": lambda: attn.moe_kv_attention(heads, kv, block_table, offsets, kv_lens, 0.1, out, None, ws, stream=stream),
            "norm": lambda: attn.moe_rms_norm(x, norm, 1e-6, out, stream=stream),
            "rotary": lambda: attn.moe_rotary(heads, pos, table, out, stream=stream),
            "append": lambda: attn.moe_latent_append(want[:, 0], s.qr[:, 0], slots, to, ws, stream=stream),
        }.get(what, lambda: attn.moe_linear_fp8(x, w, out, ws, stream=stream))
    want_out, here = call()
    here()
    out, there = call()
    errors = []

    def go():
        try:
            there()
        except Exception as e:                             # noqa: BLE001
            errors.append(e)
    t = threading.Thread(target=go)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors and torch.equal(out, want_out) and moe.moe_check_device_status(ws) == 0


@pytest.mark.parametrize("heads,latent", [(16, 512), (96, 256), (5, 512)])
def test_a_workspace_for_many_requests_serves_steps_of_fewer(heads, latent):
    """More tokens than requests, in a workspace made for as many of either: that step's units are others, and its parts larger."""
    cache = attn.LatentCache.empty(1, latent, 64)
    ws = attn.alloc_workspace(64, 64, heads, cache)
    for kv, n in (([5000] * 4, [3, 1, 4, 2]), ([700] * 62, [2] + [1] * 61), ([9000], [2]), ([300] * 64, [1] * 64), ([20000], [64])):
        s = Step(kv, n, heads, latent, 64, seed=75)
        out, lse = s.run(ws=ws)
        want, want_lse = s.run()
        assert moe.moe_check_device_status(ws) == 0
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_block_tables_from_two_host_threads():
    """Of 4,000 and of 8,192 requests, whose kernels take different amounts of shared memory; through the C ABI, as above."""
    L = attn.lib()
    calls, keep = [], []
    for B in (4000, 8192):
        ctx, new, head = i32([17] * B), i32([1] * B), i32([0])
        free = torch.arange(2 * B, dtype=torch.int32, device="cuda")
        i = dict(dtype=torch.int32, device="cuda")
        out = [torch.zeros(B, 2, **i), torch.zeros(B, **i), torch.zeros(B + 1, **i), torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(B, **i),
               torch.zeros(1, **i)]
        ws, stream = torch.zeros(512, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
        keep.append((ctx, new, head, free, out, ws, stream))
        args = (ctx.data_ptr(), new.data_ptr(), B, B, 16, free.data_ptr(), 2 * B, head.data_ptr(), out[0].data_ptr(), 2, *[t.data_ptr() for t in out[1:]],
                ws.data_ptr(), 512, stream.cuda_stream)
        calls.append(lambda args=args: L.moe_kv_build_tables(*args))
    torch.cuda.synchronize()
    statuses = [[], []]
    start = threading.Barrier(2)

    def go(i):
        torch.zeros(1, device="cuda")
        start.wait()
        for _ in range(4000):
            statuses[i].append(calls[i]())
    threads = [threading.Thread(target=go, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [{v: st.count(v) for v in set(st)} for st in statuses] == [{moe.MOE_OK: 4000}] * 2
    for ctx, _, _, _, out, ws, _ in keep:
        assert moe.moe_check_device_status(ws) == 0 and torch.equal(out[1], ctx + 1)


@pytest.mark.parametrize("T,heads,st,sh", [(4, 2, 384, 256), (4, 2, 1016, 128), (3, 4, 2048, 512), (2, 3, 128, 256), (5, 3, 136, 1000), (1, 3, 0, 128), (3, 1, 128, 0)])
def test_rotary_of_outputs_that_lie_between_one_another(T, heads, st, sh):
    """Any strides by which rows of 128 values share none, and nothing is written between them."""
    g = gen(T * heads + st)
    q, pos, table = normal(g, T, heads, 128), torch.arange(T, dtype=torch.int32, device="cuda") * 1000, attn.RotaryTable.make(128)
    span = (T - 1) * st + (heads - 1) * sh + 128
    buf = Guarded((span,), torch.bfloat16)
    out = buf.t.as_strided((T, heads, 128), (st, sh, 1))
    attn.moe_rotary(q, pos, table, out)
    buf.check()
    want, bound = ref.rotary(q, pos, table.turns)
    within(out, want, bound)
    rest = torch.ones(span, dtype=torch.bool, device="cuda")
    for t in range(T):
        for h in range(heads):
            rest[t * st + h * sh: t * st + h * sh + 128] = False
    assert (buf.t[rest].view(torch.uint8) == 0xA5).all()


def test_norm_over_its_input():
    """One row, whatever its distance to the next; several where they lie H apart; otherwise a refusal, and nothing is written."""
    g = gen(76)
    x, w = normal(g, 5, 272), normal(g, 256)
    want = torch.empty(5, 256, dtype=torch.bfloat16, device="cuda")
    attn.moe_rms_norm(x[:, :256], w, 1e-6, want)
    one = x[2:3].clone()
    attn.moe_rms_norm(one[:, :256], w, 1e-6, one[:, :256])
    assert torch.equal(one[0, :256], want[2]) and torch.equal(one[0, 256:], x[2, 256:])
    near = x[:, :256].contiguous()
    attn.moe_rms_norm(near, w, 1e-6, near)
    assert torch.equal(near, want)
    wide = x.clone()
    with pytest.raises(moe.MoEError):
        attn.moe_rms_norm(wide[:, :256], w, 1e-6, wide.view(-1)[:5 * 256].view(5, 256))
    assert torch.equal(wide, x)
