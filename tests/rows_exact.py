"""Inputs of the experts that are built by hand, for tests."""
import numpy as np

from oracle import awq_oracle as o


def words(q):
    """Codes [N, K] to the artefact's int32 words, eight per word."""
    s = np.arange(0, 32, 4, dtype=np.uint32)
    w = np.bitwise_or.reduce(q.reshape(q.shape[0], -1, 8).astype(np.uint32) << s, axis=-1).astype(np.uint32).view(np.int32)
    assert np.array_equal(o.unpack_words(w), q)
    return w
