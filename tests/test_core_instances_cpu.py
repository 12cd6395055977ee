"""The list of kernel instances that the GPU tests run is the planners' whole choice: shapes drawn with
other seeds find no other."""
import core_instances


def test_other_draws_find_no_other_instance():
    known = core_instances.instances()
    print(len(known), "instances")
    assert not set(core_instances.instances(seed=1, draws=10000)) - set(known)
