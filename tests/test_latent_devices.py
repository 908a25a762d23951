"""Refusals of tensors on another device than the call's, without a GPU: CPU
tensors that say they are on one, and a library that only notes its calls."""
import itertools

import pytest
import torch

from sparse_attention_top_idx_gb300 import dsaidx, latent

BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64


class On(torch.Tensor):
    """A CPU tensor that claims a CUDA device."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index


def on(index, *shape, dtype=BF):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
    t.index = index
    return t


class Library:
    """Notes the calls that would have been made."""

    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        return lambda *args: self.made.append(name) or 0


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(dsaidx, "_lib", lib)
    monkeypatch.setattr(latent, "_bound", lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return lib


def plan(d):
    return latent.RopePlan(on(d, 32, dtype=I64), 1.0)


def cache(d):
    return latent.LatentCache(on(d, 2, 64, latent.RECORD))


# name of a call -> (the call of its arguments, {argument: it on a device})
CALLS = {
    "rope": (lambda x, positions, plan, out: latent.rope(x, positions, plan, out=out),
             dict(x=lambda d: on(d, 3, 2, 64), positions=lambda d: on(d, 3, dtype=I64), plan=plan,
                  out=lambda d: on(d, 3, 2, 64))),
    "append": (lambda cache, c, k_pe, positions, slots, plan, status:
               latent.latent_append(cache, c, k_pe, positions, slots, plan, status=status),
               dict(cache=cache, c=lambda d: on(d, 3, 512), k_pe=lambda d: on(d, 3, 64),
                    positions=lambda d: on(d, 3, dtype=I64), slots=lambda d: on(d, 3, dtype=I64), plan=plan,
                    status=lambda d: on(d, 1, dtype=I32))),
    "slots": (lambda cache, ql, qp, slots, out, ws, lse:
              latent.latent_attend_slots(cache, ql, qp, slots, 0.1, out, ws, lse=lse),
              dict(cache=cache, ql=lambda d: on(d, 3, 16, 512), qp=lambda d: on(d, 3, 16, 64),
                   slots=lambda d: on(d, 3, 8, dtype=I64), out=lambda d: on(d, 3, 16, 512),
                   ws=lambda d: on(d, 256, dtype=torch.uint8), lse=lambda d: on(d, 3, 16, dtype=torch.float32))),
    "paged": (lambda cache, ql, qp, table, lens, out, ws, lse:
              latent.latent_attend_paged(cache, ql, qp, table, lens, 8, 0.1, out, ws, lse=lse),
              dict(cache=cache, ql=lambda d: on(d, 3, 16, 512), qp=lambda d: on(d, 3, 16, 64),
                   table=lambda d: on(d, 3, 1, dtype=I32), lens=lambda d: on(d, 3, dtype=I32),
                   out=lambda d: on(d, 3, 16, 512), ws=lambda d: on(d, 256, dtype=torch.uint8),
                   lse=lambda d: on(d, 3, 16, dtype=torch.float32))),
    "expanded": (lambda q, k, k_pe, v, cuq, cuk, out, lse, status:
                 latent.latent_attend_expanded(q, k, k_pe, v, cuq, cuk, 0.1, out, lse=lse, status=status),
                 dict(q=lambda d: on(d, 3, 2, 192), k=lambda d: on(d, 5, 2, 128), k_pe=lambda d: on(d, 5, 64),
                      v=lambda d: on(d, 5, 2, 128), cuq=lambda d: on(d, 2, dtype=I32), cuk=lambda d: on(d, 2, dtype=I32),
                      out=lambda d: on(d, 3, 2, 128), lse=lambda d: on(d, 3, 2, dtype=torch.float32),
                      status=lambda d: on(d, 1, dtype=I32))),
}


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_the_current_device_are_made(name, library):
    call, args = CALLS[name]
    call(**{k: make(0) for k, make in args.items()})
    assert len(library.made) == 1


@pytest.mark.parametrize("name,other", [(n, a) for n, (_, args) in CALLS.items() for a in args])
def test_one_argument_elsewhere_is_refused(name, other, library):
    call, args = CALLS[name]
    for here, there in itertools.permutations((0, 1)):
        with pytest.raises(ValueError, match="cuda:"):
            call(**{k: make(there if k == other else here) for k, make in args.items()})
    assert not library.made


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_a_device_that_is_not_current_are_refused(name, library):
    call, args = CALLS[name]
    with pytest.raises(ValueError, match="current"):
        call(**{k: make(1) for k, make in args.items()})
    assert not library.made


@pytest.mark.parametrize("name,other", [(n, a) for n, (_, args) in CALLS.items() for a in args if a != "plan" and a != "cache"])
def test_cpu_tensors_are_refused(name, other, library):
    call, args = CALLS[name]
    made = {k: make(0) for k, make in args.items()}
    made[other] = made[other].as_subclass(torch.Tensor)
    with pytest.raises(TypeError):
        call(**made)
    assert not library.made


def test_streams_of_another_device_are_refused(library):
    class Stream:
        device_index, cuda_stream = 1, 0
    x = on(0, 3, 2, 64)
    with pytest.raises(ValueError, match="stream"):
        latent.rope(x, on(0, 3, dtype=I64), plan(0), stream=Stream())
    assert not library.made
