"""Sizes of the operators' workspaces, and refusals of strides, on the CPU."""
import ctypes

import pytest

from stft_mel_spectrogram_amd import _native as N


@pytest.mark.parametrize("backward", [0, 1])
def test_attention_workspace_does_not_look_at_pointers_and_strides(backward):
    """A size can be asked for before there are tensors: whatever the fields hold."""
    def size(**kw):
        a = N.AttentionArgs()
        v = dict(dtype=N.FM_BF16, table_dtype=N.FM_BF16, far=8, num_buckets=4, batch=2, heads=4, kv_heads=2,
                 q_len=5, k_len=9000, head_dim=64, scale=0.125)
        v.update(kw)
        for name, value in v.items():
            setattr(a, name, value)
        return N.lib.fm_attention_workspace(ctypes.byref(a), backward)

    want = size()
    assert want > 0
    fields = [f"{t}_stride_{x}" for t in ("q", "k", "v", "o", "grad_o", "grad_q", "grad_k", "grad_v")
              for x in ("entry", "head", "time")]
    assert size(**{f: -(1 << 40) for f in fields}) == want
    assert size(**{f: 1 for f in ("q", "k", "v", "table", "bucket_map", "o", "lse", "grad_o", "grad_q")}) == want
    assert size(scale=0.0) == N.FM_E_INVAL


@pytest.mark.parametrize("kw", [dict(inner=-1), dict(inner=1 << 31), dict(inner=2, outer=-8), dict(inner=2, stride=-8),
                                dict(inner=0, stride=-8)])
def test_strided_scores_refuse(kw):
    P = 1 << 20  # an address that must not be touched
    a = dict(stride=100, inner=2, outer=400)
    a.update(kw)
    at = (P, a["stride"], a["inner"], a["outer"], P, 64)
    assert N.lib.fm_token_logprobs_strided(*at, P, P, P, P, P, P, 4, 100, 5, N.FM_F32, None) == N.FM_E_INVAL
    assert b"token log probabilities" in N.lib.fm_last_error()
    assert N.lib.fm_token_logprobs_backward_strided(*at, P, P, P, P, P, P, P, 4, 100, 5, N.FM_F32,
                                                    None) == N.FM_E_INVAL
