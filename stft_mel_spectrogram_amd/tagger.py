"""Example: a small model on top of the mel frames that tags every frame.

``python -m stft_mel_spectrogram_amd.tagger`` trains it on synthetic signals
(sequences of tones in noise; the tag of a frame is the tone that sounds) and
then tags a signal frame by frame against key and value caches; with
``--student`` it then trains a recurrent one from the first one's best tags and
runs that frame by frame, one state per channel.

It strings the package's operators together the way a program would: mel
frames -> layer norm -> blocks of attention with a learned relative position
bias and a two-layer network, each behind a layer norm -> the tags' log
probabilities with entropy and the best alternatives; with mixer="recurrence"
the blocks are a gated recurrence and a two-layer network, each behind an RMS
norm that adds the residual.  Tags can be restricted and biased while they are
read off.  Plain matrix products and the optimizer are torch's.
"""
from __future__ import annotations

import argparse
import math

import torch
from torch import nn

from . import (MelSpectrogram, adjust_logits, gated_recurrence, layer_norm, relative_attention, relative_buckets,
               rms_norm, token_logprobs, topk_distillation)


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


class ResidualNorm(nn.Module):
    """RMS norm of x plus the residual, and that sum."""

    def __init__(self, width: int):
        super().__init__()
        self.weight = nn.Parameter(torch.ones(width))

    def forward(self, x, residual):
        return (rms_norm(x, self.weight), x) if residual is None else rms_norm(x, self.weight, residual)


class RecurrentBlock(nn.Module):
    """Takes the last layer's output and the residual before it, gives its own."""

    def __init__(self, width: int):
        super().__init__()
        self.norm1, self.norm2 = ResidualNorm(width), ResidualNorm(width)
        self.into, self.out = nn.Linear(width, 3 * width), nn.Linear(width, width)
        self.up, self.down = nn.Linear(width, 4 * width), nn.Linear(4 * width, width)
        with torch.no_grad():  # memories of three to some hundred frames
            self.into.bias[width:2 * width] = torch.linspace(1.0, 6.0, width)

    def forward(self, x, residual=None, lengths=None, state=None):
        y, residual = self.norm1(x, residual)
        x, forget, gate = self.into(y).chunk(3, -1)  # slices of the projection as it lies
        h, _ = gated_recurrence(x, forget, gate, state, lengths=lengths, out_state=state)
        y, residual = self.norm2(self.out(h), residual)
        return self.down(torch.nn.functional.gelu(self.up(y))), residual


def tag_bits(tags, count: int, device="cuda"):
    """The given tags of `count` as a mask of allowed ones (int32 words)."""
    words = [0] * ((count + 31) // 32)
    for t in tags:
        if not 0 <= t < count:
            raise ValueError(f"tags must be in [0, {count}), got {t}")
        words[t // 32] |= 1 << t % 32
    return torch.tensor([w - (1 << 32) if w >> 31 else w for w in words], dtype=torch.int32, device=device)


class Tagger(nn.Module):
    """Tags of mel frames; causal, so that it can also run frame by frame."""

    def __init__(self, tags: int = 16, width: int = 128, heads: int = 4, blocks: int = 2,
                 buckets: int = 32, distance: int = 128, device="cuda", mixer: str = "attention", **mel_args):
        super().__init__()
        if mixer not in ("attention", "recurrence"):
            raise ValueError(f"mixer must be 'attention' or 'recurrence', got {mixer!r}")
        self.recurrent = mixer == "recurrence"
        mel_args = dict(sample_rate=16000, n_fft=400, hop_length=160, n_mels=80) | mel_args
        device = torch.empty(0, device=device).device  # with its index
        self.mel = MelSpectrogram(device=device, **mel_args)
        self.norm_in = Norm(self.mel.n_mels)
        self.norm_out = ResidualNorm(width) if self.recurrent else Norm(width)
        self.into = nn.Linear(self.mel.n_mels, width)
        self.blocks = nn.ModuleList(RecurrentBlock(width) if self.recurrent else Block(width, heads, buckets)
                                    for _ in range(blocks))
        self.head = nn.Linear(width, tags)
        self.to(device)
        self.bucket_map = relative_buckets(buckets, distance, bidirectional=False, device=device)

    def frames(self, signal):
        """Normalised log mel frames [batch, frames, n_mels] of [batch, samples]."""
        m = self.mel(signal).clamp_min(1e-10).log10().transpose(1, 2).contiguous()
        return self.norm_in(m)

    def logits(self, frames, lengths=None, caches=None, offset=0):
        x = self.into(frames)
        if self.recurrent:
            residual = None
            for i, block in enumerate(self.blocks):
                x, residual = block(x, residual, lengths, None if caches is None else caches[i])
            return self.head(self.norm_out(x, residual)[0])
        for i, block in enumerate(self.blocks):
            x = block(x, self.bucket_map, lengths, None if caches is None else caches[i], offset)
        return self.head(self.norm_out(x))

    def loss(self, signal, tags, lengths=None):
        """Mean negative log probability of the tags [batch, frames] (negative
        tags are left out) and the mean entropy."""
        r = token_logprobs(self.logits(self.frames(signal), lengths), tags)
        count = (tags >= 0).sum()
        return -r.logprobs.sum() / count, (r.entropy * (tags >= 0)).sum() / count

    def distill_loss(self, signal, teacher, top_k: int = 8, temperature: float = 1.0, rest: bool = False):
        """Mean distance of the frames' tags from a teacher's best top_k."""
        with torch.no_grad():
            logits = teacher.logits(teacher.frames(signal))
            asked = torch.full(logits.shape[:-1], -1, dtype=torch.int64, device=logits.device)
            best = token_logprobs(logits, asked, top_k)
        return topk_distillation(self.logits(self.frames(signal)), best.top_ids, best.top_logprobs,
                                 temperature=temperature, rest=rest).mean()

    def new_caches(self, batch: int, positions: int):
        """What `stream` keeps: keys and values, or one state per channel."""
        p = self.head.weight
        if self.recurrent:
            return [p.new_zeros((batch, p.shape[1]), dtype=torch.float32) for _ in self.blocks]
        shape = (batch, self.blocks[0].heads, positions, p.shape[1] // self.blocks[0].heads)
        return [(p.new_empty(shape), p.new_empty(shape)) for _ in self.blocks]

    @torch.no_grad()
    def stream(self, frames, top_k: int = 3, allowed=None, bias_ids=None, bias=None):
        """Frame by frame: (tags, log probabilities) of the best alternatives,
        [batch, frames, top_k].  allowed: a mask of tags as tag_bits makes it;
        bias_ids int64 and bias float32 [batch, n] are added to tags' logits."""
        b, t, _ = frames.shape
        caches = self.new_caches(b, t)
        asked = torch.full((b,), -1, dtype=torch.int64, device=frames.device)
        ids, lps = [], []
        for i in range(t):
            logits = self.logits(frames[:, i:i + 1], caches=caches, offset=i)[:, 0]
            if allowed is not None or bias is not None:
                logits = adjust_logits(logits, allowed=allowed, bias_ids=bias_ids, bias=bias)
            r = token_logprobs(logits, asked, top_k)
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
          device="cuda", report=None, mixer: str = "attention", teacher=None):
    """Trains a Tagger, from the tags or from a teacher's best ones; returns it
    and the losses."""
    torch.manual_seed(seed)
    model = Tagger(device=device, mixer=mixer)
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    frames = model.mel.out_frames(int(seconds * 16000))
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for i in range(steps):
        x, tags = tone_batch(batch, seconds, 16, frames, gen, device)
        if teacher is None:
            loss, entropy = model.loss(x, tags)
        else:
            loss = model.distill_loss(x, teacher)
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if report and i % 10 == 0:
            report(f"step {i}: loss {losses[-1]:.3f}" +
                   (f", entropy {entropy.item():.3f}" if teacher is None else ""))
    return model, losses


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description="train a small frame tagger and run it frame by frame")
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--mixer", choices=("attention", "recurrence"), default="attention")
    ap.add_argument("--student", action="store_true",
                    help="then train a recurrent tagger from the first one's best tags")
    a = ap.parse_args(argv)

    def run(name, **how):
        model, losses = train(a.steps, report=lambda s: print(s, flush=True), **how)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(1)
        frames = model.mel.out_frames(16000)
        x, tags = tone_batch(2, 1.0, 16, frames, gen)
        with torch.no_grad():
            ids, lps = model.stream(model.frames(x))
        ok = (ids[..., 0] == tags)[tags >= 0].float().mean().item()
        print(f"{name}loss {losses[0]:.3f} -> {losses[-1]:.3f}; frame by frame {100 * ok:.0f}% of the tags, "
              f"mean log probability {lps[..., 0].mean().item():.3f}")
        return model

    teacher = run("", mixer=a.mixer)
    if a.student:
        run("student: ", mixer="recurrence", teacher=teacher)


if __name__ == "__main__":
    main()
