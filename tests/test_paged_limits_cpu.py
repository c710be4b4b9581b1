"""The paged-cache operators where what a call allows ends, without a GPU."""

from test_paged_cpu import A, INVALID, OK, _attend


def test_a_bound_above_the_tokens(lib):
    """A fixed bound is clipped to the tokens that there are, before what else is asked of it."""
    so = lib.load_library()
    for most in (1, 64, 65, 2 ** 40):
        assert _attend(so, tokens=0, most=most, starts=A) == OK, most
        assert _attend(so, tokens=0, most=most, starts=A, masks=A) == OK, most
        assert _attend(so, tokens=0, most=most) == INVALID          # without starts it is tokens / batch
    for kw in (dict(tokens=6, most=0), dict(tokens=6, most=-1), dict(tokens=0, most=-1), dict(tokens=-1, most=3),
               dict(tokens=65, most=65, masks=A), dict(tokens=65, most=100, masks=A)):
        assert _attend(so, starts=A, **kw) == INVALID, kw
        assert so.rope_last_error()
