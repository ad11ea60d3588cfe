"""The binding of the operators around the attention, without a GPU."""
import types

from exact_io_aware_26_gb300 import ops


def test_a_call_whose_plan_was_dropped_is_made_all_the_same(monkeypatch):
    """Another thread may register the plan that empties the table, or change the library,
    between a call's registration and its run: the call is registered again, never lost."""
    made = []

    class Dropping:
        def run(self, op, tensors, scalars):
            if len(made) < 3:
                return None
            return ("done",)

        def register(self, *a):
            made.append(a)

    monkeypatch.setattr(ops, "_launch", Dropping())
    device = types.SimpleNamespace(index=0)
    monkeypatch.setattr(ops, "load", lambda: types.SimpleNamespace(fa_kv4_append=ops.ctypes.CFUNCTYPE(None)(lambda: None)))
    got = ops._call(ops._APPEND, (None,), (), None, lambda *a: (device, [], [], [], None))
    assert got == ("done",) and len(made) == 3
