"""Example: a small model on top of the mel frames that tags every frame.

``python -m stft_mel_spectrogram_amd.tagger`` trains it on synthetic signals
(sequences of tones in noise; the tag of a frame is the tone that sounds) and
then tags a signal frame by frame against key and value caches.

It strings the package's operators together the way a program would: mel
frames -> layer norm -> blocks of attention with a learned relative position
bias and a two-layer network, each behind a layer norm -> the tags' log
probabilities with entropy and the best alternatives.  Plain matrix products
and the optimizer are torch's.
"""
from __future__ import annotations

import argparse
import math

import torch
from torch import nn

from . import (MelSpectrogram, layer_norm, relative_attention, relative_buckets, token_logprobs)


class Norm(nn.Module):
    def __init__(self, width: int):
        super().__init__()
        self.weight = nn.Parameter(torch.ones(width))
        self.bias = nn.Parameter(torch.zeros(width))

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias)


class Block(nn.Module):
    def __init__(self, width: int, heads: int, buckets: int):
        super().__init__()
        self.heads = heads
        self.norm1, self.norm2 = Norm(width), Norm(width)
        self.qkv = nn.Linear(width, 3 * width)
        self.table = nn.Parameter(torch.zeros(buckets, heads))
        self.out = nn.Linear(width, width)
        self.up, self.down = nn.Linear(width, 4 * width), nn.Linear(4 * width, width)

    def forward(self, x, bucket_map, lengths=None, cache=None, offset=0):
        b, t, c = x.shape
        qkv = self.qkv(self.norm1(x)).view(b, t, 3 * self.heads, c // self.heads).transpose(1, 2)
        q, k, v = qkv.chunk(3, dim=1)  # slices of the projection as it lies
        if cache is not None:
            # new positions join the cache; `offset` of them were there before
            cache[0][:, :, offset:offset + t], cache[1][:, :, offset:offset + t] = k, v
            k, v = cache[0][:, :, :offset + t], cache[1][:, :, :offset + t]
        o = relative_attention(q, k, v, self.table, bucket_map, causal=True, key_lengths=lengths,
                               query_offset=offset)
        x = x + self.out(o.transpose(1, 2).reshape(b, t, c))
        return x + self.down(torch.nn.functional.gelu(self.up(self.norm2(x))))


class Tagger(nn.Module):
    """Tags of mel frames; causal, so that it can also run frame by frame."""

    def __init__(self, tags: int = 16, width: int = 128, heads: int = 4, blocks: int = 2,
                 buckets: int = 32, distance: int = 128, device="cuda", **mel_args):
        super().__init__()
        mel_args = dict(sample_rate=16000, n_fft=400, hop_length=160, n_mels=80) | mel_args
        device = torch.empty(0, device=device).device  # with its index
        self.mel = MelSpectrogram(device=device, **mel_args)
        self.norm_in, self.norm_out = Norm(self.mel.n_mels), Norm(width)
        self.into = nn.Linear(self.mel.n_mels, width)
        self.blocks = nn.ModuleList(Block(width, heads, buckets) for _ in range(blocks))
        self.head = nn.Linear(width, tags)
        self.to(device)
        self.bucket_map = relative_buckets(buckets, distance, bidirectional=False, device=device)

    def frames(self, signal):
        """Normalised log mel frames [batch, frames, n_mels] of [batch, samples]."""
        m = self.mel(signal).clamp_min(1e-10).log10().transpose(1, 2).contiguous()
        return self.norm_in(m)

    def logits(self, frames, lengths=None, caches=None, offset=0):
        x = self.into(frames)
        for i, block in enumerate(self.blocks):
            x = block(x, self.bucket_map, lengths, None if caches is None else caches[i], offset)
        return self.head(self.norm_out(x))

    def loss(self, signal, tags, lengths=None):
        """Mean negative log probability of the tags [batch, frames] (negative
        tags are left out) and the mean entropy."""
        r = token_logprobs(self.logits(self.frames(signal), lengths), tags)
        count = (tags >= 0).sum()
        return -r.logprobs.sum() / count, (r.entropy * (tags >= 0)).sum() / count

    def new_caches(self, batch: int, positions: int):
        p = self.head.weight
        shape = (batch, self.blocks[0].heads, positions, p.shape[1] // self.blocks[0].heads)
        return [(p.new_empty(shape), p.new_empty(shape)) for _ in self.blocks]

    @torch.no_grad()
    def stream(self, frames, top_k: int = 3):
        """Frame by frame: (tags, log probabilities) of the best alternatives,
        [batch, frames, top_k]."""
        b, t, _ = frames.shape
        caches = self.new_caches(b, t)
        asked = torch.full((b,), -1, dtype=torch.int64, device=frames.device)
        ids, lps = [], []
        for i in range(t):
            r = token_logprobs(self.logits(frames[:, i:i + 1], caches=caches, offset=i)[:, 0], asked, top_k)
            ids.append(r.top_ids)
            lps.append(r.top_logprobs)
        return torch.stack(ids, 1), torch.stack(lps, 1)


def tone_batch(batch: int, seconds: float, tags: int, frames: int, generator, device="cuda",
               sample_rate: int = 16000):
    """Signals of tones that change every quarter of a second, in noise, and the
    tag of each frame; the last frames of every other signal are unlabelled."""
    n = int(seconds * sample_rate)
    step = sample_rate // 4
    pick = torch.randint(0, tags, (batch, n // step + 1), generator=generator, device=device)
    tone = pick.repeat_interleave(step, 1)[:, :n]
    hz = 200.0 * 2.0 ** (tone.double() * 4.5 / tags)
    phase = torch.cumsum(hz, 1) * (2 * math.pi / sample_rate)
    x = 0.3 * phase.sin() + 0.05 * torch.randn(batch, n, generator=generator, device=device)
    at = (torch.arange(frames, device=device) * n // frames).clamp(max=n - 1)
    labels = tone[:, at].clone()
    labels[1::2, frames - frames // 8:] = -1
    return x.float(), labels


def train(steps: int = 60, batch: int = 8, seconds: float = 2.0, seed: int = 0, lr: float = 2e-3,
          device="cuda", report=None):
    """Trains a Tagger; returns it and the losses."""
    torch.manual_seed(seed)
    model = Tagger(device=device)
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    frames = model.mel.out_frames(int(seconds * 16000))
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for i in range(steps):
        x, tags = tone_batch(batch, seconds, 16, frames, gen, device)
        loss, entropy = model.loss(x, tags)
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if report and i % 10 == 0:
            report(f"step {i}: loss {losses[-1]:.3f}, entropy {entropy.item():.3f}")
    return model, losses


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description="train a small frame tagger and run it frame by frame")
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args(argv)
    model, losses = train(a.steps, report=lambda s: print(s, flush=True))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    frames = model.mel.out_frames(16000)
    x, tags = tone_batch(2, 1.0, 16, frames, gen)
    with torch.no_grad():
        ids, lps = model.stream(model.frames(x))
    ok = (ids[..., 0] == tags)[tags >= 0].float().mean().item()
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}; frame by frame {100 * ok:.0f}% of the tags, "
          f"mean log probability {lps[..., 0].mean().item():.3f}")


if __name__ == "__main__":
    main()
