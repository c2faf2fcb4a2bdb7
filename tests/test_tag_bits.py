"""The example's mask of allowed tags."""
import pytest

torch = pytest.importorskip("torch")


def test_bits():
    from stft_mel_spectrogram_amd.tagger import tag_bits
    assert tag_bits([], 5, "cpu").tolist() == [0]
    assert tag_bits([0, 4, 4], 5, "cpu").tolist() == [0b10001]
    assert tag_bits([31, 32, 63], 64, "cpu").tolist() == [-(1 << 31), 1 - (1 << 31)]


@pytest.mark.parametrize("tags,count", [([-1], 32), ([-33], 64), ([5], 5), ([40], 33), ([64], 64)])
def test_tags_that_are_none(tags, count):
    """-1 allowed the last tag of 32, and the others nothing, without a word."""
    from stft_mel_spectrogram_amd.tagger import tag_bits
    with pytest.raises(ValueError, match="tag"):
        tag_bits(tags, count, "cpu")
