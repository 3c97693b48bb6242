"""How weights reach the product over an 8-bit cache where rows are few: an fp16 value in three e5m2 terms."""
import torch


def test_three_terms_hold_an_fp16_weight():
    """Exactly from 2^-6 to 2^15 (three digits a term, each term's remainder half of its last digit at most: two terms leave
    three of eleven; from 2^-6 on an fp16 value is a multiple of 2^-16, e5m2's smallest step), and within 2^-17, half of
    that step, below."""
    u = torch.arange(1, 0x7C00, dtype=torch.int32).to(torch.int16).view(torch.float16)
    u = u[u <= 2.0 ** 15].double()
    left = u.clone()
    for _ in range(3):
        left = left - left.to(torch.float8_e5m2).double()
        assert torch.equal(left, left.to(torch.float16).double())  # (a remainder is an fp16 value again)
    assert bool((left[u >= 2.0 ** -6] == 0).all()) and float(left.abs().max()) <= 2.0 ** -17
