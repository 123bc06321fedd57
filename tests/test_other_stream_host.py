"""What the ctypes binding allocates for a call on a stream that is not the current one,
run without a GPU: a stand-in library, CPU tensors in place of device tensors, and
PyTorch's stream functions replaced by recorders."""
import contextlib

import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4


class _FakeLib:
    def __getattr__(self, name):
        return (lambda *a: 1 << 16) if name == "w4_workspace_bytes" else (lambda *a: w4.W4_OK)


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def seen(monkeypatch):
    """(stream an allocation was made under, streams it was recorded on) of every allocation."""
    made, now = [], [None]

    @contextlib.contextmanager
    def on(s):
        before, now[0] = now[0], s.cuda_stream
        yield
        now[0] = before

    def recorder(make):
        def f(*a, **k):
            t = make(*a, **k)
            t._recorded = []
            made.append((now[0], t._recorded))
            return t
        return f

    monkeypatch.setattr(w4, "_lib", _FakeLib())
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a, **k: _Stream(7))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: _Stream(h))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: self._recorded.append(s.cuda_stream))
    monkeypatch.setattr(torch, "empty", recorder(torch.empty))
    monkeypatch.setattr(torch, "zeros", recorder(torch.zeros))
    return made


def _calls():
    """Every entry point that allocates, with all it can allocate left to it."""
    M, K, N, E, T, g = 4, 256, 64, 2, 4, 128
    i8, i32, f16, bf16, f32, u8 = torch.int8, torch.int32, torch.float16, torch.bfloat16, torch.float32, torch.uint8
    z = torch.zeros
    q, sx, qw, sw = z((M, K), dtype=i8), z(M), z((K // 8, N), dtype=i32), z((K // g, N), dtype=f16)
    x, qe, se, off = z((T, K), dtype=bf16), z((E, N, K // 8), dtype=i32), z((E, N, K // g), dtype=f16), z(E + 1, dtype=i32)
    tab, ts, ro = z((N, K // 2), dtype=u8), z((N, K // g)), z((T, 2), dtype=i32)
    return {
        "w4_quant_act_per_token": (2, lambda s: w4.w4_quant_act_per_token(x, stream=s)),
        "w4a8_gemm": (2, lambda s: w4.w4a8_gemm(q, sx, qw, sw, g, stream=s)),
        "w4a8_gemm_bf16in": (3, lambda s: w4.w4a8_gemm_bf16in(x, qw, sw, g, stream=s)),
        "w4a8_gemm_noalloc": (1, lambda s: w4.w4a8_gemm_noalloc(q, sx, qw, sw, g, stream=s)),
        "w4a8_group_partials": (2, lambda s: w4.w4a8_group_partials(q, qw, g, stream=s)),
        "w4a16_gemm": (1, lambda s: w4.w4a16_gemm(x, qw, sw, g, stream=s)),
        "w4afp8_moe_grouped_gemm": (2, lambda s: w4.w4afp8_moe_grouped_gemm(z((M, K), dtype=u8), sx, off, qe, se, g, stream=s)),
        "w4_moe_route": (6, lambda s: w4.w4_moe_route(z((T, E)), 1, stream=s)),
        "w4_moe_gather_quant_fp8": (2, lambda s: w4.w4_moe_gather_quant_fp8(x, z(6, dtype=i32), stream=s)),
        "w4afp8_moe_gemm_bf16in": (3, lambda s: w4.w4afp8_moe_gemm_bf16in(x, None, off, qe, se, g, stream=s)),
        "w4_moe_silu_mul_quant_fp8": (2, lambda s: w4.w4_moe_silu_mul_quant_fp8(x, stream=s)),
        "w4_moe_combine": (1, lambda s: w4.w4_moe_combine(x, z((T, 2)), ro, stream=s)),
        "w4_quantize_groupwise": (3, lambda s: w4.w4_quantize_groupwise(x, g, stream=s)),
        "w4_repack_s4_to_uint4b8": (1, lambda s: w4.w4_repack_s4_to_uint4b8(tab, stream=s)),
        "w4_embedding_gather": (1, lambda s: w4.w4_embedding_gather(z(3, dtype=i32), tab, ts, ts, g, stream=s)),
        "w4_lm_head_gemv": (1, lambda s: w4.w4_lm_head_gemv(x, tab, ts, ts, g, stream=s)),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_allocations_belong_to_the_calls_stream(seen, name):
    count, call = _calls()[name]
    inputs = len(seen)
    call(_Stream(5))
    made = [m for m in seen[inputs:] if m[0] is not None]
    assert len(made) == count
    assert all(under == 5 for under, _ in made)
    # outputs are recorded on the caller's stream; the workspace is the call's alone
    ws = name in ("w4a8_gemm", "w4a8_gemm_bf16in", "w4a8_group_partials", "w4afp8_moe_grouped_gemm", "w4_moe_route",
                  "w4afp8_moe_gemm_bf16in")
    assert sum(r == [7] for _, r in made) == count - ws
    assert sum(r == [] for _, r in made) == ws


@pytest.mark.parametrize("name", list(_calls()))
def test_allocations_on_the_current_stream_are_plain(seen, name):
    for s in (None, _Stream(7)):
        _, call = _calls()[name]
        call(s)
    assert all(under is None and not r for under, r in seen)


def test_apply_weights_copies_on_the_calls_stream(seen, monkeypatch):
    under = []
    reshape, now = torch.Tensor.reshape, torch.cuda.stream

    @contextlib.contextmanager
    def on(s):
        under.append(s.cuda_stream)
        with now(s):
            yield
        under.pop()

    at_copy = []
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.Tensor, "reshape", lambda self, *a: (at_copy.append(list(under)), reshape(self, *a))[1])
    x = torch.zeros((2, 2, 256), dtype=torch.bfloat16).transpose(0, 1)
    w4.apply_weights(x, torch.zeros((32, 64), dtype=torch.int32), torch.zeros((2, 64), dtype=torch.float16), 128,
                     stream=_Stream(5))
    assert at_copy[0] == [5]
