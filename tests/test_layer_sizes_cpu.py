"""Sizes at the ends of what the recurrent layer's C calls accept: counts that stay within 32 bits, and refusals
beyond.  Nothing here reaches a launch."""
import pytest

import kimi_delta_attention_chunk_gb300 as kda
from kimi_delta_attention_chunk_gb300 import build as kbuild
from tests.test_layer_abi_cpu import INVALID_ARG, UNSUPPORTED, at, scan

MOST_TOKENS = 2 ** 31 - 65536 - 1


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def test_convolution_runs_at_the_most_tokens(lib):
    W, C = 4, 8
    row = C * (W + 1) * 4                                # a run's partial sums
    # one block of channels: three fillings of 152 SMs by three blocks, each a run, up to a rounding of their length
    for T in (2 ** 30, 2 ** 31 - 2 ** 25, MOST_TOKENS - 10 ** 6, MOST_TOKENS):
        need = lib.kda_short_conv_bwd_workspace_size(1, T, C, W)
        assert need % row == 0 and 3 * 152 * 3 - 8 <= need // row <= 3 * 152 * 3, T
    assert lib.kda_short_conv_bwd_workspace_size(1, MOST_TOKENS + 1, C, W) == 0


def test_scan_runs_at_the_most_tokens(lib):
    C, S = 8, 8
    for T in (2 ** 30, 2 ** 31 - 2 ** 25, MOST_TOKENS - 10 ** 6, MOST_TOKENS):
        # 96 runs: their end states, sums of step sizes, and whether a sequence begins inside
        assert lib.kda_ssm_scan_fwd_workspace_size(1, T, C, 1, S, 1, 0) == 96 * (C * S + C) * 4 + 96 * 4, T
    assert lib.kda_ssm_scan_fwd_workspace_size(1, MOST_TOKENS + 1, C, 1, S, 1, 0) == 0


def test_number_of_sequences(lib):
    """As many as tokens: offsets and histories are counted past the number in steps of a grid."""
    many = MOST_TOKENS + 1

    def conv(N, cu=at(4)):
        return lib.kda_short_conv_fwd(at(1), 8, at(2), None, 0, 1, None, cu, 1 if cu else N, 64 if cu else 0, 8, 4, N, at(3), None, None)

    def conv_bwd(N):
        return lib.kda_short_conv_bwd(at(1), 8, at(2), None, 0, 1, None, at(4), 1, 64, 8, 4, N, at(5), None, 1, at(6), at(7), None, None,
                                      at(8), 1 << 30, None)
    for N in (many, 2 ** 31 - 1):
        assert conv(N) == INVALID_ARG and conv(N, None) == INVALID_ARG and conv_bwd(N) == INVALID_ARG
        assert scan(lib, N=N, cu=at(7), G=1, ldb=16, ldc=16) == INVALID_ARG
        assert lib.kda_ssm_scan_fwd_workspace_size(1, 4096, 256, 2, 16, N, 1) == 0
        assert lib.kda_ssm_scan_bwd_workspace_size(1, 64, 256, 2, 16, N, 1) == 0
    assert lib.kda_ssm_scan_fwd_workspace_size(1, 4096, 256, 2, 16, MOST_TOKENS, 1) > 0


def test_rows_with_slots(lib):
    """Every row's slot is compared with those before it: a number of rows whose square stays small."""
    most = 1 << 18

    def conv(N, P, slots):
        return lib.kda_short_conv_step(at(1), 8, at(2), None, 0, 1, at(3), slots, P, N, 8, 4, at(5), None, None)

    def ssm(N, P, slots):
        return lib.kda_ssm_step(at(1), 8, at(2), 8, at(3), at(4), 8, at(5), 8, None, None, 0, None, 0, 1, at(6), slots, P, N, 8, 1, 8, at(8),
                                None, None)

    def step(N):
        return lib.kda_recurrent_step_slots(at(1), at(4), at(5), at(6), at(7), 1, 0.0, at(2), at(3), 8, N, 1, 128, 128, at(8), 0, None, None)
    for P in (8, 1 << 20):
        assert conv(most + 1, P, at(4)) == UNSUPPORTED and ssm(most + 1, P, at(7)) == UNSUPPORTED
    assert step(most + 1) == UNSUPPORTED
    assert conv(most, 8, at(4, 1)) == INVALID_ARG and ssm(most, 8, at(7, 1)) == INVALID_ARG      # so many are looked at
