"""Fused STFT -> mel-spectrogram forward pass for AMD MI355X (gfx950).

The compute lives in libfm.so (C ABI in include/fm.h); `MelSpectrogram` is a
thin torch-facing caller of it, and so are the operators of the models on top
of the mel frames: layer norm, RMS norm with the residual, attention with a learned
relative position bias, a gated linear recurrence, token log probabilities and
distillation from a larger model's, each with its backward pass, and logits
adjusted before a token is chosen.  Importing the package does not load the
library; touching one of its names does, and fails loudly if it is missing.
"""

_NAMES = {
    "MelSpectrogram": "melspec",
    "layer_norm": "norm",
    "layer_norm_forward": "norm",
    "layer_norm_backward": "norm",
    "relative_buckets": "attention",
    "relative_attention": "attention",
    "relative_attention_forward": "attention",
    "relative_attention_backward": "attention",
    "TokenLogprobs": "scores",
    "token_logprobs": "scores",
    "token_logprobs_forward": "scores",
    "token_logprobs_backward": "scores",
    "gated_recurrence": "recurrence",
    "gated_recurrence_forward": "recurrence",
    "gated_recurrence_backward": "recurrence",
    "rms_norm": "rmsnorm",
    "rms_norm_forward": "rmsnorm",
    "rms_norm_backward": "rmsnorm",
    "rms_norm_quantized": "rmsnorm",
    "topk_distillation": "distillation",
    "topk_distillation_forward": "distillation",
    "topk_distillation_backward": "distillation",
    "adjust_logits": "adjust",
}

__all__ = list(_NAMES)


def __getattr__(name):
    if name in _NAMES:
        import importlib
        value = getattr(importlib.import_module("." + _NAMES[name], __name__), name)
        globals()[name] = value
        return value
    raise AttributeError(name)
