"""What the binding of the recurrent layer's operators hands to the library, and what it refuses: the library is
replaced by a recorder and the tensors have no memory, so that every size can be tried."""
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from kimi_delta_attention_chunk_gb300 import kda as binding


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 16 if name.endswith("workspace_size") else 0
        return call

    def names(self):
        return [n for n, _ in self.calls if not n.endswith("workspace_size")]


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(binding, "_lib", rec)
    monkeypatch.setattr(binding, "_here", lambda *tensors: 0)
    monkeypatch.setattr(binding, "_stream_of", lambda dev: 0)
    return rec


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def f(*shape):
    return t(*shape, dtype=torch.float32)


def i(*shape):
    return t(*shape, dtype=torch.int32)


def test_single_token_calls_take_one_row_a_sequence(lib):
    N, C, G, S = 2, 16, 1, 8
    kda.short_conv_step(t(N, C), t(N, 3, C), f(C, 4))
    kda.ssm_step(t(N, C), t(N, C), f(C, S), t(N, G, S), t(N, G, S), f(N, C, S))
    kda.ssm_step(t(N, C), t(N, C), f(C, S), t(N, G, S), t(N, G, S), f(N, C, S), z=t(N, C))
    done = lib.names()
    assert done == ["kda_short_conv_step", "kda_ssm_step", "kda_ssm_step"]
    for x in (t(N, 3, C), t(N, 1, C), t(C)):
        with pytest.raises(ValueError, match=r"\[N, 16\]"):
            kda.short_conv_step(x, t(x.shape[0], 3, C), f(C, 4))
    for lead in ((N, 3), (N, 1), ()):
        u, v = t(*lead, C), t(*lead, G, S)
        with pytest.raises(ValueError, match=r"\[N, 16\]"):
            kda.ssm_step(u, u, f(C, S), v, v, f(u.shape[0], C, S))
    with pytest.raises(ValueError):                      # the groups without their states
        kda.ssm_step(t(N, C), t(N, C), f(C, S), t(N, S), t(N, S), f(N, C, S))
    assert lib.names() == done


def test_prompts_take_batches_of_rows(lib):
    C, S = 16, 8
    for lead in ((5,), (1, 5, 2)):
        u, v = t(*lead, C), t(*lead, 1, S)
        with pytest.raises(ValueError):
            kda.short_conv_fwd(u, f(C, 4))
        with pytest.raises(ValueError):
            kda.short_conv_bwd(u, f(C, 4), u)
        with pytest.raises(ValueError):
            kda.ssm_scan_fwd(u, u, f(C, S), v, v)
        with pytest.raises(ValueError):
            kda.ssm_scan_bwd(u, u, f(C, S), v, v, u)
    assert lib.names() == []


MANY = 2 ** 32 + 3      # three, in the library's 32 bits


def test_sizes_past_the_librarys_integers(lib):
    C, S = 1, 8
    calls = [
        lambda: kda.short_conv_fwd(t(1, MANY, C), f(C, 4)),
        lambda: kda.short_conv_fwd(t(MANY, 1, C), f(C, 4)),
        lambda: kda.short_conv_fwd(t(1, 8, MANY), f(MANY, 4)),
        lambda: kda.short_conv_fwd(t(1, 8, C), f(C, 4), cu_seqlens=i(MANY)),
        lambda: kda.short_conv_bwd(t(1, MANY, C), f(C, 4), t(1, MANY, C)),
        lambda: kda.short_conv_step(t(MANY, C), t(MANY, 3, C), f(C, 4)),
        lambda: kda.short_conv_step(t(2, C), t(MANY, 3, C), f(C, 4), slots=i(2)),
        lambda: kda.ssm_step(t(MANY, C), t(MANY, C), f(C, S), t(MANY, 1, S), t(MANY, 1, S), f(MANY, C, S)),
        lambda: kda.ssm_step(t(2, C), t(2, C), f(C, S), t(2, 1, S), t(2, 1, S), f(MANY, C, S), slots=i(2)),
        lambda: kda.ssm_scan_fwd(t(1, MANY, C), t(1, MANY, C), f(C, S), t(1, MANY, 1, S), t(1, MANY, 1, S)),
        lambda: kda.ssm_scan_fwd(t(1, 8, C), t(1, 8, C), f(C, S), t(1, 8, 1, S), t(1, 8, 1, S), cu_seqlens=i(MANY)),
        lambda: kda.ssm_scan_bwd(t(1, MANY, C), t(1, MANY, C), f(C, S), t(1, MANY, 1, S), t(1, MANY, 1, S), t(1, MANY, C)),
        lambda: kda.recurrent_step(t(2, 1, 64), t(2, 1, 64), t(2, 1, 64), t(2, 1, 64), t(2, 1), f(MANY, 1, 64, 64), slots=i(2)),
        lambda: kda.pages_alloc(i(MANY), 5),
        lambda: kda.pages_alloc(i(8), MANY),
        lambda: kda.pages_free(i(MANY), i(5)),
        lambda: kda.pages_fork(i(4, MANY), i(4), i(8), i(2), i(2), 16),
        lambda: kda.pages_fork(i(MANY, 4), i(MANY), i(8), i(2), i(2), 16),
        lambda: kda.pages_fork(i(4, 4), i(4), i(MANY), i(2), i(2), 16),
        lambda: kda.pages_fork(i(4, 4), i(4), i(8), i(MANY), i(MANY), 16),
        lambda: kda.pages_fork(i(4, 4), i(4), i(8), i(2), i(2), MANY),
        lambda: kda.pages_compact(i(MANY)),
        lambda: kda.pages_copy(f(MANY, 4), i(2), i(2)),
        lambda: kda.pages_copy(f(8, 4), i(MANY), i(MANY)),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(ValueError, match="2\\*\\*31"):
            call()
        assert lib.calls == [], k
    kda.pages_free(i(8), i(MANY))                        # any number of entries: counted in 64 bits
    assert lib.calls[-1][1][3] == MANY
