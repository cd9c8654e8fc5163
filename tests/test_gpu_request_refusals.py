"""What the Python entry points of the operators for many requests refuse when the tensors are on the
device (MI355X): every check raises before anything is enqueued, and the same call
with none of the faults works. Then what autograd sees of them, and their streams."""
import pytest
import torch

import bit_quantized_gemm_amd as w4

DEV = "cuda:0"
BF, F16, F32, I32, I64 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.int64
pytestmark = pytest.mark.gpu


def zeros(*shape, dtype=BF, device=DEV):
    return torch.zeros(shape, dtype=dtype, device=device)


def every_other(*shape, dtype=BF):
    """A tensor of this shape whose last dimension is not dense."""
    return zeros(*shape[:-1], 2 * shape[-1], dtype=dtype)[..., ::2]


def host(*shape, dtype=BF):
    return zeros(*shape, dtype=dtype, device="cpu")


def norm_args():
    return dict(x=zeros(2, 3, 40), y=zeros(2, 3, 40), gate=zeros(2, 1, 40), post_norm=True, post_weight=zeros(40), weight=zeros(40), bias=zeros(40),
                scale=zeros(40), shift=zeros(2, 3, 40))


def adapt_args():
    return dict(y=zeros(5, 24), x=zeros(5, 64), down=zeros(3, 4, 64), up=zeros(3, 4, 24), adapter=zeros(5, dtype=I32),
                scaling=zeros(3, dtype=F32), ranks=zeros(3, dtype=I32))


def append_args():
    return dict(k=zeros(4, 2, 16), v=zeros(4, 2, 16), k_cache=zeros(3, 8, 2, 16), v_cache=zeros(3, 8, 2, 16), slots=torch.arange(4, device=DEV))


def packed_args():
    return dict(q=zeros(9, 4, 16), k=zeros(9, 2, 16), v=zeros(9, 2, 16), starts=torch.tensor([0, 4, 9], dtype=I32, device=DEV))


def paged_args():
    return dict(q=zeros(2, 1, 4, 16), k_cache=zeros(5, 16, 2, 16), v_cache=zeros(5, 16, 2, 16), table=zeros(2, 3, dtype=I32),
                lens=torch.tensor([20, 3], dtype=I32, device=DEV))


CALLS = {"block_norm": norm_args, "lora_adapters": adapt_args, "cache_append": append_args, "packed_attention": packed_args,
         "paged_attention": paged_args}
FAULTS = [
    ("block_norm", TypeError, dict(x=lambda: zeros(2, 3, 40, dtype=F32))), ("block_norm", TypeError, dict(x=3)),
    ("block_norm", ValueError, dict(x=lambda: host(2, 3, 40))), ("block_norm", ValueError, dict(x=lambda: zeros(40))),
    ("block_norm", ValueError, dict(x=lambda: every_other(2, 3, 40))), ("block_norm", TypeError, dict(y=lambda: zeros(2, 3, 40, dtype=F16))),
    ("block_norm", ValueError, dict(y=lambda: zeros(2, 1, 40))), ("block_norm", ValueError, dict(y=lambda: host(2, 3, 40))),
    ("block_norm", TypeError, dict(gate=lambda: zeros(40, dtype=F32))), ("block_norm", ValueError, dict(gate=lambda: zeros(2, 40))),
    ("block_norm", ValueError, dict(gate=lambda: zeros(2, 3, 1))), ("block_norm", ValueError, dict(gate=lambda: zeros(1, 2, 3, 40))),
    ("block_norm", ValueError, dict(scale=lambda: every_other(2, 3, 40))), ("block_norm", ValueError, dict(shift=lambda: host(40))),
    ("block_norm", ValueError, dict(weight=lambda: zeros(41))), ("block_norm", ValueError, dict(bias=lambda: zeros(1, 40))),
    ("block_norm", ValueError, dict(weight=lambda: every_other(40))), ("block_norm", TypeError, dict(post_weight=lambda: zeros(40, dtype=F16))),
    ("block_norm", ValueError, dict(kind="group")), ("block_norm", ValueError, dict(kind=None)), ("block_norm", TypeError, dict(eps="small")),
    ("block_norm", w4.GemmError, dict(eps=0.0)), ("block_norm", w4.GemmError, dict(residual_scale=float("nan"))),
    ("block_norm", ValueError, dict(y=None)), ("block_norm", ValueError, dict(y=None, gate=None, post_norm=False, post_weight=None, residual_scale=2.0)),
    ("block_norm", ValueError, dict(y=None, gate=None, post_norm=False, post_weight=None, residual=lambda: zeros(2, 3, 40))),
    ("block_norm", ValueError, dict(post_norm=False)), ("block_norm", ValueError, dict(out=lambda: zeros(2, 3, 41))),
    ("block_norm", TypeError, dict(residual=lambda: zeros(2, 3, 40, dtype=F16))), ("block_norm", w4.GemmError, dict(out=lambda: zeros(3, 40).expand(2, 3, 40))),
    ("lora_adapters", TypeError, dict(y=lambda: zeros(5, 24, dtype=F32))), ("lora_adapters", ValueError, dict(y=lambda: host(5, 24))),
    ("lora_adapters", ValueError, dict(y=lambda: zeros(5, 1, 24))), ("lora_adapters", TypeError, dict(x=lambda: zeros(5, 64, dtype=F16))),
    ("lora_adapters", ValueError, dict(x=lambda: zeros(6, 64))), ("lora_adapters", ValueError, dict(x=lambda: every_other(5, 64))),
    ("lora_adapters", ValueError, dict(down=lambda: zeros(3, 64))), ("lora_adapters", ValueError, dict(down=lambda: zeros(3, 4, 63))),
    ("lora_adapters", ValueError, dict(down=lambda: zeros(4, 3, 64).transpose(0, 1))), ("lora_adapters", ValueError, dict(up=lambda: zeros(3, 5, 24))),
    ("lora_adapters", TypeError, dict(up=lambda: zeros(3, 4, 24, dtype=F16))), ("lora_adapters", TypeError, dict(adapter=lambda: zeros(5, dtype=I64))),
    ("lora_adapters", ValueError, dict(adapter=lambda: zeros(4, dtype=I32))), ("lora_adapters", ValueError, dict(adapter=lambda: host(5, dtype=I32))),
    ("lora_adapters", TypeError, dict(scaling=lambda: zeros(3))), ("lora_adapters", ValueError, dict(ranks=lambda: zeros(2, dtype=I32))),
    ("lora_adapters", ValueError, dict(out=lambda: zeros(5, 25))), ("lora_adapters", ValueError, dict(out=lambda: every_other(5, 24))),
    ("lora_adapters", w4.GemmError, dict(out=lambda: zeros(24).expand(5, 24))),
    ("lora_adapters", w4.GemmError, dict(x=lambda: zeros(5, 60), down=lambda: zeros(3, 4, 60))),
    ("lora_adapters", w4.GemmError, dict(down=lambda: zeros(3, 129, 64), up=lambda: zeros(3, 129, 24))),
    ("cache_append", TypeError, dict(k=lambda: zeros(4, 2, 16, dtype=F32))), ("cache_append", ValueError, dict(k=lambda: host(4, 2, 16))),
    ("cache_append", ValueError, dict(v=lambda: zeros(4, 3, 16))), ("cache_append", TypeError, dict(k_cache=lambda: zeros(3, 8, 2, 16, dtype=F16))),
    ("cache_append", ValueError, dict(k_cache=lambda: zeros(24, 2, 16))), ("cache_append", ValueError, dict(v_cache=lambda: zeros(4, 8, 2, 16))),
    ("cache_append", ValueError, dict(k_cache=lambda: zeros(3, 8, 2, 24), v_cache=lambda: zeros(3, 8, 2, 24))),
    ("cache_append", TypeError, dict(slots=lambda: zeros(4, dtype=I32))), ("cache_append", ValueError, dict(slots=lambda: zeros(5, dtype=I64))),
    ("cache_append", ValueError, dict(v=lambda: every_other(4, 2, 16))), ("cache_append", ValueError, dict(slots=lambda: host(4, dtype=I64))),
    ("cache_append", w4.GemmError, dict(k_cache=lambda: zeros(8, 2, 16).expand(3, 8, 2, 16))),
    ("packed_attention", TypeError, dict(q=lambda: zeros(9, 4, 16, dtype=F32))), ("packed_attention", ValueError, dict(q=lambda: host(9, 4, 16))),
    ("packed_attention", ValueError, dict(q=lambda: zeros(1, 9, 4, 16))), ("packed_attention", ValueError, dict(k=lambda: zeros(8, 2, 16))),
    ("packed_attention", TypeError, dict(v=lambda: zeros(9, 2, 16, dtype=F16))), ("packed_attention", ValueError, dict(v=lambda: every_other(9, 2, 16))),
    ("packed_attention", TypeError, dict(starts=lambda: zeros(3, dtype=I64))), ("packed_attention", ValueError, dict(starts=lambda: zeros(0, dtype=I32))),
    ("packed_attention", ValueError, dict(starts=lambda: host(3, dtype=I32))), ("packed_attention", ValueError, dict(out=lambda: zeros(9, 4, 8))),
    ("packed_attention", w4.GemmError, dict(q=lambda: zeros(9, 3, 16))), ("packed_attention", w4.GemmError, dict(scale=-1.0)),
    ("packed_attention", w4.GemmError, dict(v=lambda: zeros(1, 2, 16).expand(9, 2, 16))),
    ("paged_attention", TypeError, dict(q=lambda: zeros(2, 1, 4, 16, dtype=F32))), ("paged_attention", ValueError, dict(q=lambda: host(2, 1, 4, 16))),
    ("paged_attention", ValueError, dict(q=lambda: zeros(2, 4, 16))), ("paged_attention", ValueError, dict(q=lambda: zeros(2, 1, 4, 24))),
    ("paged_attention", TypeError, dict(k_cache=lambda: zeros(5, 16, 2, 16, dtype=F16))), ("paged_attention", ValueError, dict(v_cache=lambda: zeros(5, 16, 1, 16))),
    ("paged_attention", TypeError, dict(table=lambda: zeros(2, 3, dtype=I64))), ("paged_attention", ValueError, dict(table=lambda: zeros(3, 3, dtype=I32))),
    ("paged_attention", ValueError, dict(table=lambda: zeros(2, dtype=I32))), ("paged_attention", ValueError, dict(table=lambda: every_other(2, 3, dtype=I32))),
    ("paged_attention", ValueError, dict(table=lambda: host(2, 3, dtype=I32))), ("paged_attention", TypeError, dict(lens=lambda: zeros(2, dtype=I64))),
    ("paged_attention", ValueError, dict(lens=lambda: zeros(3, dtype=I32))), ("paged_attention", ValueError, dict(out=lambda: zeros(2, 1, 4, 8))),
    ("paged_attention", w4.GemmError, dict(k_cache=lambda: zeros(5, 8, 2, 16), v_cache=lambda: zeros(5, 8, 2, 16))),
    ("paged_attention", w4.GemmError, dict(scale=0.0))]


@pytest.mark.parametrize("name,error,over", FAULTS, ids=[f"{n}-{'-'.join(o)}-{i}" for i, (n, _, o) in enumerate(FAULTS)])
def test_refused(name, error, over):
    args = {**CALLS[name](), **{k: v() if callable(v) else v for k, v in over.items()}}
    with pytest.raises(error):
        getattr(w4, name)(**args)


@pytest.mark.parametrize("name", CALLS)
def test_accepted(name):
    getattr(w4, name)(**CALLS[name]())
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", CALLS)
def test_nothing_to_do(name):
    """Empty batches, sequences and caches: results of the right shape, nothing enqueued."""
    empty = {"block_norm": dict(x=zeros(2, 0, 40), y=zeros(2, 0, 40), shift=zeros(2, 0, 40)),
             "lora_adapters": dict(y=zeros(0, 24), x=zeros(0, 64), adapter=zeros(0, dtype=I32)),
             "cache_append": dict(k=zeros(0, 2, 16), v=zeros(0, 2, 16), slots=zeros(0, dtype=I64)),
             "packed_attention": dict(q=zeros(0, 4, 16), k=zeros(0, 2, 16), v=zeros(0, 2, 16)),
             "paged_attention": dict(q=zeros(0, 1, 4, 16), table=zeros(0, 3, dtype=I32), lens=zeros(0, dtype=I32))}[name]
    r = getattr(w4, name)(**{**CALLS[name](), **empty})
    assert (r[0] if isinstance(r, tuple) else r).shape[:2] == {"block_norm": (2, 0), "lora_adapters": (0, 24), "cache_append": (3, 8),
                                                               "packed_attention": (0, 4), "paged_attention": (0, 1)}[name]


# ---------------------------------------------------------------- autograd and streams

@pytest.mark.parametrize("name", CALLS)
def test_autograd(name):
    """Results are detached whatever the inputs require; a tensor given as an output has changed in place."""
    args = CALLS[name]()
    first = {"block_norm": "x", "lora_adapters": "x", "cache_append": "k", "packed_attention": "q", "paged_attention": "q"}[name]
    args[first] = args[first].requires_grad_()
    outs = {"block_norm": ("out", "residual"), "cache_append": ("k_cache", "v_cache")}.get(name, ("out",))
    shape = args["y"].shape if name == "lora_adapters" else args[first].shape
    given = {k: args.get(k, torch.zeros(shape, dtype=BF, device=DEV)) for k in outs}
    was = [t._version for t in given.values()]
    r = getattr(w4, name)(**{**args, **given})
    assert [t._version for t in given.values()] == [v + 1 for v in was]
    assert not any(t.requires_grad for t in (r if isinstance(r, tuple) else (r,)))
    if name != "cache_append":
        r = getattr(w4, name)(**args)
        assert not any(t.requires_grad for t in (r if isinstance(r, tuple) else (r,)))


@pytest.mark.parametrize("name", CALLS)
def test_handle_that_the_native_step_sees(name, monkeypatch):
    seen = []

    class Recorder:
        def __getattr__(self, fn):
            return lambda *args: seen.append((fn, torch._C._cuda_getCurrentRawStream(0)))

    monkeypatch.setattr(w4._native, "binding", lambda: Recorder())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = torch.cuda.Stream()
        for stream, want in ((None, side), (0, torch.cuda.default_stream()), (torch.cuda.default_stream(), torch.cuda.default_stream()),
                             (other, other), (other.cuda_stream, other)):
            getattr(w4, name)(**CALLS[name](), stream=stream)
            assert seen.pop() == (name, want.cuda_stream), stream


def test_outside_of_torch_inference_mode():
    with torch.inference_mode():
        for name, args in CALLS.items():
            getattr(w4, name)(**args())
