"""The counter-based generator of dropout against the published vectors of Philox 4x32 of 10 rounds (Salmon et al. 2011), of any counter
and key, and the tests' form of it, which starts at group 0, against that (no GPU)."""
import random

import pytest

import recur_ref

LOW = (1 << 32) - 1


def philox(counter, key):
    c, k = list(counter), list(key)
    for _ in range(10):
        high0, low0 = divmod(c[0] * 0xD2511F53, 1 << 32)
        high1, low1 = divmod(c[2] * 0xCD9E8D57, 1 << 32)
        c = [high1 ^ c[1] ^ k[0], low1, high0 ^ c[3] ^ k[1], low0]
        k = [(k[0] + 0x9E3779B9) & LOW, (k[1] + 0xBB67AE85) & LOW]
    return c


@pytest.mark.parametrize("counter,key,want", [
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([LOW] * 4, [LOW] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0], [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_published_vectors(counter, key, want):
    assert philox(counter, key) == want


def test_words_of_a_call():
    """Counter (group, number of the call), key the seed, both little end first, two's complement."""
    rng = random.Random(1)
    for seed, call in [(0, 0), (-1, -1), (1 << 62, -(1 << 63))] + [(rng.getrandbits(63), rng.getrandbits(63)) for _ in range(20)]:
        words = recur_ref.words(seed, call, 11)
        halves = lambda v: [v & LOW, (v >> 32) & LOW]  # noqa: E731
        assert words == [w for group in range(3) for w in philox([group, 0] + halves(call), halves(seed))][:11]
