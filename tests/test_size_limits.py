"""Sizes at the ends of the kernels' index arithmetic are refused on the host (no GPU: nothing is launched)."""
import ctypes

INT_MAX = 2 ** 31 - 1


def test_the_recurrence_refuses_more_rows_than_its_rounds_number():
    """The last round's end has to be an int; B = 0 does nothing, after the sizes' checks."""
    from bwd_la_fwd_gb300 import la
    lib = la.load_library()

    def forward(N, B=1):
        return lib.la_gated_scan(0x10000, 0x1000000000000, None, 0x2000000000000, None, B, N, 8, 0, 1, None, None)

    def backward(N, B=1):
        return lib.la_gated_scan_backward(*((k + 1) << 48 for k in range(4)), None, None, 5 << 48, 6 << 48, None, B, N, 8, 0,
                                          1, None, None)

    for f in (forward, backward):
        assert f(INT_MAX) == 1 and f(INT_MAX - 1023) == 1
        assert f(INT_MAX, B=0) == 1 and f(INT_MAX - 1024, B=0) == 0


def test_rotary_refuses_more_rows_and_heads_than_an_int_numbers():
    from bwd_la_fwd_gb300 import la
    lib = la.load_library()
    freq = (ctypes.c_ulonglong * 128)()

    def call(N, B=1, Hq=1, Hk=0):
        return lib.la_rotary(1 << 48, 2 << 48, 3 << 48, 4 << 48, freq, None, 0, 0, 0, 1.0, B, Hq, Hk, N, 8, 2, 1, None, None)

    assert call(INT_MAX) == 1 and call(INT_MAX - 1023) == 1
    assert call(INT_MAX, B=0) == 1 and call(INT_MAX - 1024, B=0) == 0
    # heads of Q and K are numbered together
    assert call(1, Hq=INT_MAX, Hk=INT_MAX) == 1 and call(1, Hq=2 ** 30) == 1 and call(1, Hq=2 ** 29, Hk=2 ** 29) == 1
    assert call(0, Hq=2 ** 29, Hk=2 ** 29 - 1) == 0
