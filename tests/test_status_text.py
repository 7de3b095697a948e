"""The text of every set of status bits: the calls of one step share a status
word, so any of them can stand in it together (no GPU)."""
import itertools

import combine_ep_plan_amd as ep

BITS = {
    ep.EP_STATUS_BAD_EXPERT: "expert id",
    ep.EP_STATUS_CAPACITY: "capacity",
    ep.EP_STATUS_BAD_REGION: "KV region",
    ep.EP_STATUS_BAD_PAGE: "page, sequence or length",
}


def test_every_set_of_bits_names_each_of_them_and_no_other():
    seen = set()
    for n in range(1, len(BITS) + 1):
        for some in itertools.combinations(BITS, n):
            text = ep.status_string(sum(some))
            for bit, word in BITS.items():
                assert (word in text) == (bit in some), (some, text)
            seen.add(text)
    assert len(seen) == 2 ** len(BITS) - 1


def test_capacity_speaks_for_pages_too():
    assert "page" in ep.status_string(ep.EP_STATUS_CAPACITY)
    assert "receive" in ep.status_string(ep.EP_STATUS_CAPACITY)


def test_other_codes_keep_their_text():
    assert ep.status_string(0) == "ok"
    assert ep.status_string(ep.EP_ERR_INVALID_ARG) == "invalid argument"
    for code in (16, 17, 31, 99, -5, 1 << 30):
        assert ep.status_string(code) == "unknown code"
