"""Which addresses sub_probs and sub_verify_sample take, on the host (no GPU needed)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def s():
    import substitute_speculative_decoding_gb300 as s
    return s


def at(x):
    return C.c_void_p(x)        # never followed: each call is refused first


def refused(s, code, word):
    return code == s.SUB_EINVAL and word in s._lib.sub_last_error()


def test_probabilities_lie_apart_from_the_logits(s):
    base = 1 << 20
    for x in (base + 4, base - 4, base + 4 * 19, base - 4 * 19):
        assert refused(s, s._probs(at(base), 2, 10, 1.0, at(x), None), b"apart")
    assert refused(s, s._probs(at(base + 2), 2, 10, 1.0, at(2 * base), None), b"aligned")
    assert refused(s, s._probs(at(base), 2, 10, 1.0, at(2 * base + 1), None), b"aligned")


def test_verification_writes_apart_from_its_inputs(s):
    size = {"p": 2 * 4 * 10, "q": 2 * 3 * 10, "draft": 2 * 3, "u": 2 * 4, "tokens": 2 * 4, "acc": 2}
    place = {k: (i + 1) << 20 for i, k in enumerate(size)}

    def call(**kw):
        a = {k: at(v) for k, v in {**place, **kw}.items()}
        return s._verify_sample(a["p"], a["q"], a["draft"], a["u"], 2, 3, 10, a["tokens"], a["acc"],
                                None)
    for out in ("tokens", "acc"):
        for other in size:
            if other == out:
                continue
            for x in (place[other], place[other] + 4 * (size[other] - 1),
                      place[other] - 4 * (size[out] - 1)):
                assert refused(s, call(**{out: x}), b"apart"), (out, other)
    for k in size:
        assert refused(s, call(**{k: place[k] + 2}), b"aligned"), k
    # sizes whose product is beyond 64 bits
    assert refused(s, s._verify_sample(at(4096), None, at(4), at(8), 1 << 24, 1 << 20, 1 << 20,
                                       at(1 << 50), at(16), None), b"apart")
